// Window attention for single tokens over a cache (tp_window_attn_decode).
//
// One query per sequence at position n - 1, n = lens[i] the sequence's keys
// in the cache: it sees the last `window` keys and the first `sinks` ones.
// Reading K and V once is the whole cost (2 G flops per byte for G query
// heads per key head, far below the ridge), so:
// * a block takes one (sequence, key head) and a slice of its visible keys;
//   the slices fill the SMs whatever the batch, and a second kernel joins
//   them by their maxima and sums;
// * the G query heads of a key head (16 at a time) are the 16 rows of an
//   m16n8k16 product, so a key is read once for all of them and the
//   arithmetic stays far from the limit;
// * every warp streams its own 16-key tiles through its own ring of three
//   cp.async stages (no block barrier in the loop) and keeps its own running
//   maximum, sum and O; the block's warps are joined at its end.  Four stages
//   or eight warps, which leave one block per SM, were 10-25% slower.
// P enters P V as the rounded value and the rounded rest, so O is off by its
// own rounding alone (with one term 1.4 times that), whatever else is in the
// batch.  Groups of up to 8 query heads leave the rows 8-15 of the product
// empty: the rests go there and cost no product of their own (32 sequences of
// 4100 visible keys, 8 key heads of 128 read by 4 heads each, in two slices: 85.0
// us; with one term and the empty rows computed 86.9).  Larger groups take a second one (16
// such sequences, groups of 16: 69.2 against 65.0 us with one term).
// Keys past the visible range are read as zeros and masked, so what the
// cache holds beyond lens never enters, whatever it is.  A sum of 0 stands for
// no key at all; the sum of a row with a NaN score is NaN, and so is its O.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "stream_mma.cuh"
#include "tp_internal.h"

namespace tp {
namespace {

constexpr int kTileKeys = 16;  // per warp and step
constexpr int kStages = 3;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;      // query heads per block
constexpr int kMaxSplits = 255;
constexpr int kFoldRows = 8;   // query heads up to which the rests of P take the rows 8-15
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

struct DecArgs {
  const void *q, *k, *v;
  const int* lens;
  void* o;
  float* lse;   // [b, heads] or nullptr
  float* po;    // partial O: [item][split][rows][d], rows = min(group, 16)
  float2* pml;  // partial (max in log2 units, sum): [item][split][rows]
  long long ldq, ldo, ldk, ldv, bsk, bsv;
  int cap, heads, kv_heads, group, gtiles, rows, splits;
  int window, sinks;
  float scale_log2;
};

template <int DH>
struct DecSmem {
  static constexpr int kStageBytes = 2 * kTileKeys * DH * 2;  // K and V of one tile
  static constexpr int kBytes = kWarps * kStages * kStageBytes;
  static_assert(kBytes >= kWarps * kRows * DH * 4 + kWarps * kRows * 8, "join area");
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF) {
    __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&t);
  }
  __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&t);
}

// Two values as the rounded pair and the rounded rest.
template <bool BF>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2<BF>(a, b);
  const float2 h = BF ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi))
                      : __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack2<BF>(a - h.x, b - h.y);
}

template <bool BF>
__device__ __forceinline__ void store1(void* p, long long i, float v) {
  if (BF)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// The visible keys of a sequence of n keys as a list: [0, ns), then
// [lo, lo + total - ns).
struct Visible {
  int ns, lo, total;
  __device__ __forceinline__ Visible(int n, const DecArgs& a) {
    n = min(max(n, 0), a.cap);
    lo = max(0, n - a.window);
    ns = min(a.sinks, lo);
    total = ns + n - lo;
  }
  __device__ __forceinline__ int key(int t) const { return t < ns ? t : lo + (t - ns); }
};

// Keys per slice: equal slices of whole block steps.
__device__ __forceinline__ int slice_keys(int total, int splits) {
  constexpr int step = kWarps * kTileKeys;
  const int per = (total + splits - 1) / splits;
  return (per + step - 1) / step * step;
}

// FOLD: at most kFoldRows query heads, row r + 8 of P holds the rest of row r.
template <bool BF, int DH, bool FOLD>
__global__ void __launch_bounds__(kThreads) window_decode(const DecArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStageBytes = DecSmem<DH>::kStageBytes;
  constexpr int kRowBytes = DH * 2, kChunks = DH / 8;
  constexpr int kTerms = FOLD ? 1 : 2;   // products of P V
  constexpr int kHalves = FOLD ? 1 : 2;  // row halves that are query heads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x, split = blockIdx.y;
  const int gt = item % a.gtiles;
  const int kvh = (item / a.gtiles) % a.kv_heads;
  const int bi = item / a.gtiles / a.kv_heads;
  const int rows = min(a.group - gt * kRows, kRows);
  const int head0 = kvh * a.group + gt * kRows;

  pdl_next();  // the join may be scheduled
  const Visible vis(a.lens[bi], a);
  const int per = slice_keys(vis.total, a.splits);
  const int t0 = min(split * per, vis.total), t1 = min(t0 + per, vis.total);

  // Q fragments: rows lane / 4 and + 8, columns 16 kk + 2 (lane % 4) and + 8.
  uint32_t qf[DH / 16][4];
  {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + bi * a.ldq + head0 * DH;
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r + 8 * (i & 1), col = 16 * kk + c + 8 * (i >> 1);
        qf[kk][i] = (i & 1) < kHalves && row < rows ? *reinterpret_cast<const uint32_t*>(q + row * DH + col) : 0u;
      }
  }

  const uint8_t* kbase = static_cast<const uint8_t*>(a.k) + (bi * a.bsk + kvh * DH) * 2;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.v) + (bi * a.bsv + kvh * DH) * 2;
  const uint32_t ring =
      static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * kStages * kStageBytes;
  constexpr int kStep = kWarps * kTileKeys;
  const int first = t0 + warp * kTileKeys;
  const int tiles = first < t1 ? (t1 - first + kStep - 1) / kStep : 0;

  // Tile i of this warp into stage i % kStages: 16-byte chunk j of key row r
  // at chunk j ^ (r & 7), so the eight rows of an ldmatrix hit eight banks groups.
  auto fetch = [&](int i) {
    const uint32_t st = ring + (i % kStages) * kStageBytes;
    const int t = first + i * kStep;
#pragma unroll
    for (int x = 0; x < kTileKeys * kChunks / 32; ++x) {
      const int id = x * 32 + lane;
      const int r = id / kChunks, j = id % kChunks;
      const bool ok = t + r < t1;
      const long long key = ok ? vis.key(t + r) : 0;
      const uint32_t dst = st + r * kRowBytes + ((j ^ (r & 7)) << 4);
      cp_async16(dst, kbase + (key * a.ldk) * 2 + j * 16, ok);
      cp_async16(dst + kTileKeys * kRowBytes, vbase + (key * a.ldv) * 2 + j * 16, ok);
    }
  };

  float o[DH / 8][4];
#pragma unroll
  for (int n = 0; n < DH / 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
  float m[kHalves], l[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.0f;
  }

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < tiles) fetch(i);
    cp_commit();
  }
  // ldmatrix source rows: lanes 0-7, 8-15, 16-23, 24-31 address the four 8 x 8
  // matrices.  K: keys 0-7 / 8-15 x columns +0 / +8; V (transposed): keys 0-7 /
  // 8-15 of two neighbouring 8-column groups.
  const int krow = (lane & 7) + ((lane >> 4) << 3), kcol = (lane >> 3) & 1;
  const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vcol = lane >> 4;
  for (int i = 0; i < tiles; ++i) {
    cp_wait<kStages - 2>();
    __syncwarp();  // every lane's copies of this stage have landed, and the
                   // stage fetched below has been read by every lane
    if (i + kStages - 1 < tiles) fetch(i + kStages - 1);
    cp_commit();
    const uint32_t sk = ring + (i % kStages) * kStageBytes;
    const uint32_t sv = sk + kTileKeys * kRowBytes;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      uint32_t b[4];
      ldmatrix4<false>(b, sk + krow * kRowBytes + (((2 * kk + kcol) ^ (krow & 7)) << 4));
      mma16816<BF>(s[0], qf[kk], b[0], b[1]);
      mma16816<BF>(s[1], qf[kk], b[2], b[3]);
    }
    // keys of this lane: t + 8 n + 2 (lane % 4) + {0, 1}
    const int t = first + i * kStep + 2 * (lane & 3);
    float mx[kHalves];
    bool up = false;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      mx[h] = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 2 * h; e < 2 * h + 2; ++e) {
          const bool in = t + 8 * n + (e & 1) < t1;
          s[n][e] = in ? s[n][e] * a.scale_log2 : -INFINITY;
          mx[h] = fmaxf(mx[h], s[n][e]);
        }
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      up = up || mx[h] > m[h];
    }
    // A tile holds at least one key, so after the first the maxima are finite
    // (for finite scores); O is rescaled only when one has risen.
    if (__any_sync(0xffffffffu, up)) {
      float f[kHalves];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const float mn = fmaxf(m[h], mx[h]);
        f[h] = m[h] == -INFINITY ? 0.0f : ex2_approx(m[h] - mn);
        m[h] = mn;
        l[h] *= f[h];
      }
#pragma unroll
      for (int n = 0; n < DH / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= f[(e >> 1) & (kHalves - 1)];
    }
    uint32_t pf[kTerms][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const float p0 = ex2_approx(s[n][2 * h] - m[h]), p1 = ex2_approx(s[n][2 * h + 1] - m[h]);
        l[h] += p0;
        l[h] += p1;
        if constexpr (FOLD)
          split2<BF>(p0, p1, pf[0][2 * n], pf[0][2 * n + 1]);
        else
          split2<BF>(p0, p1, pf[0][2 * n + h], pf[1][2 * n + h]);
      }
#pragma unroll
    for (int n = 0; n < DH / 16; ++n) {
      uint32_t b[4];
      ldmatrix4<true>(b, sv + vrow * kRowBytes + (((2 * n + vcol) ^ (vrow & 7)) << 4));
#pragma unroll
      for (int e = 0; e < kTerms; ++e) {
        mma16816<BF>(o[2 * n], pf[e], b[0], b[1]);
        mma16816<BF>(o[2 * n + 1], pf[e], b[2], b[3]);
      }
    }
  }
  cp_wait<0>();
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }

  // Join the block's warps: O, maximum and sum of each through shared memory.
  __syncthreads();  // the rings are done with
  float* so = reinterpret_cast<float*>(smem);                                 // [warp][16][DH]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * kRows * DH);          // [warp][16]
  {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < DH / 8; ++n) {
      float* d = so + (warp * kRows + r) * DH + 8 * n + c;
      if constexpr (FOLD) {
        *reinterpret_cast<float2*>(d) = make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
      } else {
        *reinterpret_cast<float2*>(d) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2*>(d + 8 * DH) = make_float2(o[n][2], o[n][3]);
      }
    }
    if ((lane & 3) == 0) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        sml[warp * kRows + r + 8 * h] = make_float2(m[h], l[h]);
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * DH; x += kThreads) {
    const int r = x / DH, c = x - r * DH;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sml[w * kRows + r].x);
    float acc = 0.0f, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * kRows + r];
      if (ml.y == 0.0f) continue;  // this warp saw no key
      const float f = ex2_approx(ml.x - mm);
      acc = fmaf(f, so[(w * kRows + r) * DH + c], acc);
      ll = fmaf(f, ml.y, ll);
    }
    if (a.splits > 1) {
      const long long p = (static_cast<long long>(item) * a.splits + split) * a.rows + r;
      a.po[p * DH + c] = acc;
      if (c == 0) a.pml[p] = make_float2(mm, ll);
    } else {
      store1<BF>(a.o, bi * a.ldo + (head0 + r) * DH + c, ll != 0.0f ? acc / ll : 0.0f);
      if (c == 0 && a.lse != nullptr)
        a.lse[static_cast<long long>(bi) * a.heads + head0 + r] =
            ll != 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    }
  }
}

// Joins the slices of one (sequence, query head): a phase of DH / 4 threads
// takes every kPhases-th slice, the phases are added in order.
template <bool BF, int DH>
__global__ void __launch_bounds__(256) window_decode_join(const DecArgs a) {
  constexpr int kLanes = DH / 4, kPhases = 256 / kLanes;
  __shared__ float s_w[kMaxSplits + 1];
  __shared__ float s_red[8];
  __shared__ float4 s_acc[kPhases][kLanes];
  const int head = blockIdx.x % a.heads, bi = blockIdx.x / a.heads;
  const int kvh = head / a.group, gh = head - kvh * a.group;
  const int item = (bi * a.kv_heads + kvh) * a.gtiles + gh / kRows;
  const long long p0 = static_cast<long long>(item) * a.splits * a.rows + gh % kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();  // the slices are complete
  // one slice per thread (splits <= 255): the common maximum, then the weights
  const float2 ml = static_cast<int>(threadIdx.x) < a.splits
                        ? a.pml[p0 + static_cast<long long>(threadIdx.x) * a.rows]
                        : make_float2(-INFINITY, 0.0f);
  float mm = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  if (lane == 0) s_red[warp] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mm = fmaxf(mm, s_red[w]);
  __syncthreads();
  const float wgt = ml.y == 0.0f ? 0.0f : ex2_approx(ml.x - mm);
  if (static_cast<int>(threadIdx.x) < a.splits) s_w[threadIdx.x] = wgt;
  float ll = wgt * ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
  if (lane == 0) s_red[warp] = ll;
  __syncthreads();
  ll = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ll += s_red[w];
  const int ph = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = ph; s < a.splits; s += kPhases) {
    const float f = s_w[s];
    const float4 v = *reinterpret_cast<const float4*>(
        a.po + (p0 + static_cast<long long>(s) * a.rows) * DH + 4 * c);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  s_acc[ph][c] = acc;
  __syncthreads();
  if (ph == 0) {
#pragma unroll
    for (int i = 1; i < kPhases; ++i) {
      const float4 v = s_acc[i][c];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + bi * a.ldo +
                                                head * DH + 4 * c);
    dst[0] = pack2<BF>(acc.x * inv, acc.y * inv);
    dst[1] = pack2<BF>(acc.z * inv, acc.w * inv);
    if (c == 0 && a.lse != nullptr)
      a.lse[static_cast<long long>(bi) * a.heads + head] =
          ll != 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
  }
}

// Slices per (sequence, key head): as many as fill the blocks that run at once
// (two per SM), rounded up, each at least kMinKeys keys; from 2 SMs of items on
// none is cut.  More and shorter ones cost more joining: one sequence of 131072
// keys, 4 key heads of 128 in bf16 (267 MB), 48 us with 74 slices, 56 with 148,
// 70 with 255; 32 sequences of 4100 visible keys, 8 key heads (537 MB): 85 us
// with two, 91 with four, 96 with five.  Rounding up starts a second round of
// blocks, which costs sequences of one length (20 and 32 of 4100 keys: 70 and 85
// us, rounded down 62 and 79) and gains more where lengths differ, since all get
// the same number of slices (20 of 1 to 8192 keys: 59 us, rounded down 95; one of
// 65536 keys among 31 of 512: 324 against 621, where the bytes alone take 51).
constexpr int kMinKeys = 256;

int plan_splits(const WindowDecode& w) {
  const int64_t gt = (w.heads / w.kv_heads + kRows - 1) / kRows;
  const int64_t items = w.b * w.kv_heads * gt;
  const int64_t keys = std::min(w.cap, w.window + w.sinks);
  const int64_t want = (2LL * sm_count() + items - 1) / items;
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({want, (keys + kMinKeys - 1) / kMinKeys, kMaxSplits})));
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <bool BF, int DH>
tp_status decode(const WindowDecode& w, void* scratch, cudaStream_t stream) {
  DecArgs a{};
  a.q = w.q;
  a.k = w.k;
  a.v = w.v;
  a.lens = w.lens;
  a.o = w.o;
  a.lse = w.lse;
  a.ldq = w.ldq;
  a.ldo = w.ldo;
  a.ldk = w.ldk;
  a.ldv = w.ldv;
  a.bsk = w.bsk;
  a.bsv = w.bsv;
  a.cap = static_cast<int>(w.cap);
  a.heads = w.heads;
  a.kv_heads = w.kv_heads;
  a.group = w.heads / w.kv_heads;
  a.gtiles = (a.group + kRows - 1) / kRows;
  a.rows = std::min(a.group, kRows);
  a.window = static_cast<int>(w.window);
  a.sinks = static_cast<int>(w.sinks);
  a.scale_log2 = w.scale * kLog2e;
  a.splits = plan_splits(w);
  const int64_t items = w.b * w.kv_heads * a.gtiles;
  const size_t ml = align256(static_cast<size_t>(items) * a.splits * a.rows * sizeof(float2));
  a.pml = static_cast<float2*>(scratch);
  a.po = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + (a.splits > 1 ? ml : 0));
  constexpr int smem = DecSmem<DH>::kBytes;
  auto kern = a.rows <= kFoldRows ? window_decode<BF, DH, true> : window_decode<BF, DH, false>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "window decode smem");
  const double keys = double(std::min(w.cap, w.window + w.sinks)) * w.b;
  LaunchScope scope(TP_KIND_ATTN_FWD, 4.0 * DH * keys * w.heads, 4.0 * DH * keys * w.kv_heads,
                    stream, a.splits > 1 ? 2 : 1);
  kern<<<dim3(static_cast<unsigned>(items), a.splits), kThreads, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess && a.splits > 1) {
    // Scheduled while the slices finish; it waits for them itself.
    e = launch_kernel(window_decode_join<BF, DH>, dim3(static_cast<unsigned>(w.b * w.heads)), 256, 0,
                      stream, true, a);
  }
  return e == cudaSuccess ? TP_OK : cuda_fail(e, "window decode launch");
}

}  // namespace

// Enough for this batch and every smaller one: n items are cut into fewer than
// 2 SMs + n slices, and into none from 2 SMs on.
size_t window_decode_scratch_bytes(const WindowDecode& w) {
  const int64_t keys = std::min(w.cap, w.window + w.sinks);
  const int64_t most = std::min<int64_t>((keys + kMinKeys - 1) / kMinKeys, kMaxSplits);
  if (most == 1) return 256;
  const int group = w.heads / w.kv_heads;
  const int64_t full = 2LL * sm_count();
  const int64_t n = std::min<int64_t>(full, w.b * w.kv_heads * ((group + kRows - 1) / kRows));
  const size_t rows =
      static_cast<size_t>(std::min(full + n - 1, n * most)) * std::min(group, kRows);
  return align256(rows * sizeof(float2)) + align256(rows * w.d * sizeof(float));
}

tp_status launch_window_decode(const WindowDecode& w, void* scratch, cudaStream_t stream) {
  if (w.dtype == TP_BF16)
    return w.d == 64 ? decode<true, 64>(w, scratch, stream) : decode<true, 128>(w, scratch, stream);
  return w.d == 64 ? decode<false, 64>(w, scratch, stream) : decode<false, 128>(w, scratch, stream);
}

}  // namespace tp
