// Attention over a sliding window with sinks on the sm_100a tensor cores:
// forward and backward (tp_window_attn_fwd / _bwd).
//
//   O = softmax(scale Q K^T) V per head, where query r of a sequence sits at
//   position p = r + sk - sq and sees key c when
//     c <= p  and  (p - c < window  or  c < sinks).
//   Query head j reads key / value head j / G, G = heads / kv_heads.
// Backward, with P the probabilities and D = rowsum(dO * O):
//   dS = P (dO V^T - D),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
//   dK and dV summed over the G query heads that share them.
//
// Same tile machinery as the full causal core (tp_attention_sm100.cu): TMA
// into 128-byte-swizzled shared memory, tcgen05 products with S, P and the
// accumulators in tensor memory, one row per thread in the softmax.  What the
// window changes:
// * Work per query tile is the key blocks of [first visible, diagonal] plus
//   the sink blocks in front of them; blocks in between are never loaded.
//   The two query tiles of a CTA share one list of blocks and each takes part
//   in those it sees.
// * A 32-column chunk a row sees whole takes the unmasked path; the others
//   (window edge, diagonal, sinks) go through a 32-bit visibility mask.
// * A row may see nothing in a block (its window starts later) or at all
//   (p < 0): the running maximum then stays -inf and P is 0, and a row that
//   saw nothing ends with O = 0 and LSE = -inf.
// * dK / dV: a key tile's queries are one contiguous range, [k0, k1 + window),
//   or everything after it where the tile holds sinks.  The heads of a group
//   follow one another in one accumulation (fixed order, no atomics).  Tiles
//   whose queries take long (sinks, wide windows, few heads) are cut along
//   (head, query) into slices with fp32 partials that a last kernel adds in
//   slice order, so no SM is left with one long tile at the end.
// * Sequences are the third dimension of the tensor maps: rows past a
//   sequence's end read as zero, never as its neighbour's values.
//
// bf16 and fp16 inputs; P and dS are rounded to the input type for their
// products (fp32 accumulation), as the products take one type for both
// operands.  In the backward, queries that see at most kSplitKeys keys give P
// and dS as two terms, the rounded value and the rounded rest, and the
// products take both (whole query tiles, and in dK / dV whole key tiles): with
// few keys the row term D, taken from the rounded O,
// already costs as much accuracy as the results' own rounding, and the
// rounding of dS would come on top (gradients 1.5-1.8 times as far from exact
// as their rounding alone, 1.1-1.4 times with the two terms).  Rows with many
// keys average the error of D out; the one rounding of P and of dS stays, and
// O and the gradients are 1.3 times as far off as their own rounding (2.1e-3
// against 1.6e-3 in bf16).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_sm100.cuh"
#include "ptx_sm100.cuh"
#include "tp_internal.h"

namespace tp {
namespace {

constexpr int kBM = 128;  // query rows per tile
constexpr int kBN = 128;  // keys per tile (dK / dV)
constexpr int kB64 = 64;  // keys per block (forward, dQ), queries per block (dK / dV)
constexpr int kThreads = 384;
constexpr float kRescaleLog2 = 8.0f;  // O keeps a stale maximum up to 2^8 behind
constexpr float kCheckSum = 255.0f;   // a row sum above this may hide such a key
constexpr int kSplitKeys = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// kind::f16 descriptor: fp16 operands, or bf16 ones.
template <bool BF>
__host__ __device__ constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn) {
  return BF ? idesc_bf16_f32(m, n, a_mn, b_mn) : idesc_f16_f32(m, n, a_mn, b_mn);
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF) {
    __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&t);
  }
  return pack_half2(a, b);
}

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two values as the rounded pair and the rounded rest.
template <bool BF>
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = pack2<BF>(v.x, v.y);
  const float2 h = unpack2<BF>(hi);
  lo = pack2<BF>(v.x - h.x, v.y - h.y);
}

// Values i and i + 1 of the four that hold them, i even.
__device__ __forceinline__ float2 half4(const float4& v, int i) {
  return (i & 2) ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
}

// Eight fp32 values as one 16-byte store of the input type.
template <bool BF>
__device__ __forceinline__ uint4 pack8t(const float* v, float f) {
  return make_uint4(pack2<BF>(v[0] * f, v[1] * f), pack2<BF>(v[2] * f, v[3] * f),
                    pack2<BF>(v[4] * f, v[5] * f), pack2<BF>(v[6] * f, v[7] * f));
}

struct WinArgs {
  int sq, sk, off;  // off = sk - sq: query r sits at position r + off
  int heads, kv_heads, group;
  int window, sinks;  // both clamped to sk
  float scale, scale_log2;
  float* lse;  // [b, heads, sq]
  // backward
  const float* nlse;  // -LSE * log2(e) and -D: [b * heads] rows of sp floats,
  const float* nd;    // zero beyond sq, 64 zeros after the last row
  int sp;
  void *dq, *dk, *dv;
  long long lddq, lddk, lddv;
  // dK / dV items: nsink_tiles key tiles hold sinks; the two classes of tiles
  // are cut into split_s and split_w slices; partials of cut tiles in part.
  int bkv, key_tiles, sink_tiles, split_s, split_w, items;
  int kv_ctas;  // persistent CTAs of the dK / dV part
  float* part;
  WaitCtl status;
};

// Key blocks of BN that some row of the query tile [r0, r0 + 128) sees
// through the window: [lo, hi], hi = -1 when the tile sees no key.  Every
// block in front of them that holds a sink is seen too.
struct Blocks {
  int lo, hi;
};

template <int BN>
__device__ __forceinline__ Blocks blocks_of(int r0, const WinArgs& a) {
  const int r1 = min(r0 + kBM, a.sq) - 1;
  Blocks b;
  const int p1 = r1 + a.off;
  if (r1 < r0 || p1 < 0) {
    b.lo = 0;
    b.hi = -1;
  } else {
    b.lo = max(0, r0 + a.off - a.window + 1) / BN;
    b.hi = p1 / BN;
  }
  return b;
}

// The CTA's list of key blocks for its two query tiles: [lo, hi], then sink
// blocks [0, ns).  Every listed block is seen by one of the tiles at least.
// With keys in front of the window, [lo, hi] runs from the diagonal down: the
// first keys that a row meets are its nearest ones, where the first block of
// the window may hide all of its keys from the last rows and send them through
// the exact maximum a block later (160 against 166 us on 8192 tokens, 32
// heads, window 1024, 4 sinks; 23 against 21 on windows of 257, five blocks
// long).  Without, it runs up from block 0, where every row sees keys and the
// two tiles end apart, so that one tile's epilogue overlaps the other's last
// blocks (73 against 81 us on 4096 tokens, 16 heads, all visible).
template <int BN>
struct BlockList {
  Blocks t0, t1;
  int nsb, ns, lo, hi, n;
  bool down;
  __device__ __forceinline__ BlockList(int r0, const WinArgs& a) {
    t0 = blocks_of<BN>(r0, a);
    t1 = blocks_of<BN>(r0 + kBM, a);
    nsb = (a.sinks + BN - 1) / BN;
    lo = t0.lo;
    hi = max(t0.hi, t1.hi);
    down = lo > 0;
    ns = hi < 0 ? 0 : min(nsb, lo);
    n = hi < 0 ? 0 : ns + hi - lo + 1;
  }
  __device__ __forceinline__ int block(int j) const {
    if (j >= n - ns) return j - (n - ns);
    return down ? hi - j : j;  // lo = 0 when it runs up
  }
  __device__ __forceinline__ bool sees(int x, int j) const {
    const int kb = block(j);
    const int xlo = x ? t1.lo : t0.lo, xhi = x ? t1.hi : t0.hi;
    return kb <= xhi && (kb >= xlo || kb < nsb);
  }
  // listed blocks that tile x sees
  __device__ __forceinline__ int count(int x) const {
    const int xlo = x ? t1.lo : t0.lo, xhi = x ? t1.hi : t0.hi;
    return xhi < 0 ? 0 : xhi + 1 - max(0, xlo - nsb);
  }
};

// Whether queries in general see at most kSplitKeys keys (by the window), so
// that P and dS are given in two terms everywhere.  Otherwise those at the
// first kSplitKeys positions do, which are the ones that see the first keys
// only.
__device__ __forceinline__ bool split_all(const WinArgs& a) {
  return a.window <= kSplitKeys - a.sinks;
}

// Visible columns of a row within one key block: [0, end) intersected with
// [first, inf) or [0, sink).
struct RowMask {
  int end, first, sink;
  // all of [c, c + 32) visible
  __device__ __forceinline__ bool full(int c) const {
    return c + 32 <= end && (c >= first || c + 32 <= sink);
  }
  // bit i: column c + i visible
  __device__ __forceinline__ uint32_t bits(int c) const {
    const uint32_t before_end = prefix(end - c);
    return before_end & (~prefix(first - c) | prefix(sink - c));
  }
  static __device__ __forceinline__ uint32_t prefix(int n) {
    return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
  }
};

// Whether all rows of a tile, positions [p0, p0 + 128), see all of the key
// block at k0.
__device__ __forceinline__ bool all_visible(int p0, int k0, const WinArgs& a) {
  return k0 + kB64 - 1 <= p0 && (k0 > p0 + kBM - 1 - a.window || k0 + kB64 <= a.sinks);
}

// Row with query position p (p < sk) in the key block that starts at k0.
__device__ __forceinline__ RowMask row_mask(int p, int k0, const WinArgs& a) {
  RowMask m;
  m.end = p + 1 - k0;
  m.first = p - a.window + 1 - k0;
  m.sink = a.sinks - k0;
  return m;
}

// The maximum raw score among a row's visible keys of one block, -inf if none.
__device__ __forceinline__ float row_max_masked(uint32_t srow, const RowMask& m) {
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < kB64; c += 32) {
    float v[32];
    tmem_ld32(srow + c, v);
    if (!m.full(c)) {
      const uint32_t vis = m.bits(c);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = ((vis >> i) & 1u) ? v[i] : -INFINITY;
    }
    mx = max32(v, mx);
  }
  return mx;
}

// P = 2^(s * scale_log2 - m) over one block row, packed in registers; returns
// the row sum of the unrounded P.  ALL: every row of the tile sees the whole
// block.  Otherwise hidden keys give 0, and a chunk that no row of the warp
// sees costs no exponential.  (Leaving the columns behind the sinks out of a
// sink block's products as well was slower in a version with blocks of 128
// keys, 196 against 188 us on the first case above.)
template <bool BF, bool ALL>
__device__ __forceinline__ float exp_row(uint32_t srow, const RowMask& mask, float scale_log2,
                                         float m, uint32_t (&pk)[kB64 / 2]) {
  const float2 sc2 = make_float2(scale_log2, scale_log2), nm2 = make_float2(-m, -m);
  float2 acc = make_float2(0.0f, 0.0f);
  // The next chunk's tensor-memory load is in flight while this one is
  // computed (one wait per chunk, after the computation).
  uint32_t nx[32];
  tmem_ld32_nowait(srow, nx);
  tmem_wait_ld(nx);
#pragma unroll
  for (int c = 0; c < kB64; c += 32) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(nx[i]);
    if (c + 32 < kB64) tmem_ld32_nowait(srow + c + 32, nx);
    const uint32_t vis = ALL ? 0xffffffffu : mask.bits(c);
    if (ALL || __any_sync(0xffffffffu, vis != 0u)) {
      float2 u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 t = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), sc2, nm2);
        u[i] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
        if (!ALL)
          u[i] = make_float2((vis >> (2 * i)) & 1u ? u[i].x : 0.0f,
                             (vis >> (2 * i + 1)) & 1u ? u[i].y : 0.0f);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[c / 2 + i] = pack2<BF>(u[i].x, u[i].y);
#pragma unroll
      for (int k = 8; k >= 1; k >>= 1)
#pragma unroll
        for (int i = 0; i < k; ++i) u[i] = __fadd2_rn(u[i], u[i + k]);
      acc = __fadd2_rn(acc, u[0]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[c / 2 + i] = 0u;
    }
    if (c + 32 < kB64) tmem_wait_ld(nx);
  }
  return acc.x + acc.y;
}

// One box per 64 columns of a [rows x DH] tile; the halves are rows * 128
// bytes apart.
template <int DH>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                          int head, int row, int seq, int rows) {
#pragma unroll
  for (int c = 0; c < DH / 64; ++c)
    tma_load_3d(dst + c * rows * 128, map, bar, head * DH + 64 * c, row, seq);
}

template <int DH>
struct FwdSmem {
  static constexpr int kStages = 4;
  static constexpr int kTile = kBM * DH * 2, kTile64 = kB64 * DH * 2;
  static constexpr int kBox = 32 * 128;  // 32 rows x 64 columns of O, per softmax warp
  // Q[2], ring of (K, V), O boxes, barriers
  static constexpr int kBytes = 1024 + 2 * kTile + 2 * kStages * kTile64 + 8 * kBox + 256;
};

// The t-th item of this CTA, or r0 = -1: rounds of one item per CTA in snake
// order, longest rows first, heads fastest.
struct FwdItem {
  int r0, head, bi;
  __device__ __forceinline__ FwdItem(int t, const WinArgs& a) {
    const long long n = gridDim.x, c = blockIdx.x;
    const long long k = t * n + ((t & 1) ? n - 1 - c : c);
    const int bh = a.bkv * a.group;
    r0 = -1;
    if (k >= a.items) return;
    const int pair = static_cast<int>(k / bh);
    const int h = static_cast<int>(k - static_cast<long long>(pair) * bh);
    r0 = 2 * kBM * (a.items / bh - 1 - pair);
    head = h % a.heads;
    bi = h / a.heads;
  }
  // whether query tile x is loaded (n: the item's blocks)
  __device__ __forceinline__ bool has_q(int x, int n, const WinArgs& a) const {
    return n > 0 && r0 + x * kBM < a.sq;
  }
};

// Persistent: a CTA per SM walks items of (sequence, head, pair of adjacent
// 128-row query tiles), warp 0 TMA, warp 1 tensor memory, warps 1 / 2 the MMA
// issue and warps 4-7 / 8-11 the softmax of tile 0 / 1.  Blocks of 64 keys, so
// that tensor memory holds two S per tile beside O: the next block's S is
// there when a block's P has been given, and the softmax does not wait for the
// products (with one S of 128 keys it did for 1740 of 4400 clocks a block).
// The ring of K and V runs on across items, a Q tile is loaded when the
// previous item's last S is done, and the next item's first two S run under an
// item's epilogue (a launch, load and epilogue of its own took 19% of an
// item of 20 blocks).
// What bounds it is the tensor pipe in the shape chosen here, not at its rate:
// with N = 64 and both operands in shared memory a product of 32 clocks holds
// the pipe for 48 (6 KB of operands), so a tile's block of 64 keys takes it 384
// clocks for S and 256 for P V, 1280 for both tiles, and a pair of blocks takes
// 1550.  Measured: 8192 tokens, 32 heads of 128, window 1024, 4 sinks (129
// GFLOP) 159 us, 810 TFLOP/s (through the Python call, one at a time, 181);
// tensor pipe active in 47% of the cycles, which is 80% of what that shape
// allows; exponentials 42%.
template <bool BF, int DH>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
               const WinArgs a) {
  using C = FwdSmem<DH>;
  constexpr int kTile = C::kTile, kTile64 = C::kTile64, kSt = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;               // [2] query tiles
  uint8_t* sKV = sQ + 2 * kTile;    // stage st: K at +0, V at +kTile64
  uint8_t* sO = sKV + kSt * 2 * kTile64;  // a box per softmax warp
  uint64_t* bars = reinterpret_cast<uint64_t*>(sO + 8 * C::kBox);
  uint64_t* kv_full = bars;          // [4] stages
  uint64_t* kv_empty = bars + 4;     // [4]
  uint64_t* s_full = bars + 8;       // [tile][buffer]: S ready
  uint64_t* p_full = bars + 12;      // [tile][buffer]: P stored (and O rescaled)
  uint64_t* o_full = bars + 16;      // [tile][buffer]: the buffer's P V done
  uint64_t* q_full = bars + 20;      // [2] tiles
  uint64_t* q_empty = bars + 22;     // [2] tiles: the item's last S done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);  // both tiles' products
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // one arrival per warp of the tile's softmax group
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, *tmem_slot);  // uniform
  // Tile x, buffer b (the parity of the block's place in the ring): S at
  // columns [256 x + 64 b, + 64), P over its first 32; O at [256 x + 128, + DH).
  auto tS = [tmem](int x, int b) { return tmem + static_cast<uint32_t>(256 * x + 64 * b); };
  auto tO = [tmem](int x) { return tmem + static_cast<uint32_t>(256 * x + 128); };
  bool ok = true;  // no wait of this thread has given up

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------- TMA producer
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmO);
      uint32_t g = 0u, nq[2] = {0u, 0u};  // blocks and query tiles loaded so far
      for (int t = 0; ok; ++t) {
        const FwdItem it(t, a);
        if (it.r0 < 0) break;
        const BlockList<kB64> bl(it.r0, a);
        auto load_q = [&](int x) {
          if (!it.has_q(x, bl.n, a)) return true;
          if (!mbar_wait(&q_empty[x], (nq[x] & 1u) ^ 1u, a.status, kStatusAttnTimeout))
            return false;
          ++nq[x];
          mbar_arrive_expect_tx(&q_full[x], kTile);
          load_tile<DH>(sQ + x * kTile, &tmQ, &q_full[x], it.head, it.r0 + x * kBM, it.bi, kBM);
          return true;
        };
        if (!(ok = load_q(0))) break;
        for (int j = 0; j < bl.n; ++j, ++g) {
          const int st = static_cast<int>(g % kSt);
          uint8_t* dst = sKV + st * (2 * kTile64);
          const int krow = bl.block(j) * kB64, kvh = it.head / a.group;
          if (!(ok = mbar_wait(&kv_empty[st], ((g / kSt) & 1u) ^ 1u, a.status,
                               kStatusAttnTimeout)))
            break;
          mbar_arrive_expect_tx(&kv_full[st], 2 * kTile64);
          load_tile<DH>(dst, &tmK, &kv_full[st], kvh, krow, it.bi, kB64);
          load_tile<DH>(dst + kTile64, &tmV, &kv_full[st], kvh, krow, it.bi, kB64);
          if (j == 0 && !(ok = load_q(1))) break;
        }
      }
    }
  } else if (warp <= 2) {
    // ---------------------------------------------------- MMA issuer of a tile
    // Per listed block j that the tile sees: P V_j; then S of block j + 2, in
    // the same buffer.  The MMAs run in issue order, so S overwrites P only
    // after its product has read it.  An issuer of its own per tile: one for
    // both was busy for 1.5 times as long as its products ran, most of it
    // waiting for one tile while the other's P was there.
    constexpr uint32_t kIdS = idesc<BF>(kBM, kB64, false, false);  // Q K^T
    constexpr uint32_t kIdO = idesc<BF>(kBM, DH, false, true);     // P V
    const int x = warp - 1;
    const uint32_t q_addr = smem_u32(sQ + x * kTile);
    uint32_t pbits = 0u;       // bit b: parity of p_full[x][b]'s next wait
    uint32_t g0 = 0u, nq = 0u;  // blocks and query tiles of the items before
    for (int t = 0; ok; ++t) {
      const FwdItem it(t, a);
      if (it.r0 < 0) break;
      const BlockList<kB64> bl(it.r0, a);
      const int total = bl.count(x);
      bool some = false;  // a P V product of this item has been issued
      int left = total;   // S products to issue
      if (it.has_q(x, bl.n, a)) {
        if (!(ok = warp_mbar_wait(&q_full[x], nq & 1u, a.status, kStatusAttnTimeout))) break;
        ++nq;
        if (total == 0) warp_umma_commit(&q_empty[x]);
      }
      for (int j = -2; j < bl.n; ++j) {
        const uint32_t g = g0 + static_cast<uint32_t>(j), gn = g + 2u;
        const int b = static_cast<int>(g & 1u);
        if (j >= 0 && bl.sees(x, j)) {
          if (!(ok = warp_mbar_wait(&p_full[2 * x + b], (pbits >> b) & 1u, a.status,
                                    kStatusAttnTimeout)))
            break;
          pbits ^= 1u << b;
          tc_fence_after();
          const uint32_t v_addr = smem_u32(sKV + (g % kSt) * (2 * kTile64) + kTile64);
          warp_umma_ts4(tO(x), tS(x, b), sw128_desc(v_addr, kB64 * 128, 1024), kIdO,
                        some ? 1u : 0u);
          warp_umma_commit(&o_full[2 * x + b]);
          some = true;
        }
        if (j >= 0) warp_umma_commit(&kv_empty[g % kSt]);
        if (j + 2 < bl.n) {
          // Waited for whether seen or not: an issuer that skipped blocks would
          // release a stage twice.
          if (!(ok = warp_mbar_wait(&kv_full[gn % kSt], (gn / kSt) & 1u, a.status,
                                    kStatusAttnTimeout)))
            break;
          if (bl.sees(x, j + 2)) {
            tc_fence_after();
            const uint32_t k_addr = smem_u32(sKV + (gn % kSt) * (2 * kTile64));
#pragma unroll
            for (int c = 0; c < DH / 64; ++c)
              warp_umma_ss4(tS(x, b), sw128_desc(q_addr + c * kBM * 128, 16, 1024),
                            sw128_desc(k_addr + c * kB64 * 128, 16, 1024), kIdS, c > 0 ? 1u : 0u);
            warp_umma_commit(&s_full[2 * x + b]);
            if (--left == 0) warp_umma_commit(&q_empty[x]);
          }
        }
      }
      g0 += static_cast<uint32_t>(bl.n);
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t orow_t = tO(x) + lane_off;
    uint8_t* box = sO + (warp - 4) * C::kBox;
    uint32_t bits = 0u;  // bit b: parity of s_full[x][b]'s next wait
    uint32_t g0 = 0u;    // blocks of the items before
    // The buffer's P V, by the parity its S had.
    auto wait_o = [&](int b) {
      const bool done = mbar_wait(&o_full[2 * x + b], ((bits >> b) & 1u) ^ 1u, a.status,
                                  kStatusAttnTimeout);
      if (done) tc_fence_after();
      return done;
    };
    for (int t = 0; ok; ++t) {
      const FwdItem it(t, a);
      if (it.r0 < 0) break;
      const BlockList<kB64> bl(it.r0, a);
      const int row0 = it.r0 + x * kBM + quarter * 32, r = row0 + lane;
      // Rows past the end take the last position: their results are not stored.
      const int p = min(r, a.sq - 1) + a.off;
      const int total = bl.count(x);
      float m_used = -INFINITY, l_run = 0.0f;
      int cnt = 0, last = 0;  // blocks so far; the buffer of the last one
      for (int j = 0; j < bl.n && cnt < total; ++j) {
        if (!bl.sees(x, j)) continue;
        const int b = static_cast<int>((g0 + j) & 1u);
        const uint32_t srow = tS(x, b) + lane_off;
        if (!(ok = mbar_wait(&s_full[2 * x + b], (bits >> b) & 1u, a.status, kStatusAttnTimeout)))
          break;
        bits ^= 1u << b;
        tc_fence_after();
        const int k0 = bl.block(j) * kB64;
        const RowMask mask = row_mask(p, k0, a);
        const bool all = all_visible(it.r0 + x * kBM + a.off, k0, a);
        // A warp none of whose rows has seen a key yet takes the exact maximum.
        const bool first = __all_sync(0xffffffffu, m_used == -INFINITY);
        if (first) m_used = row_max_masked(srow, mask) * a.scale_log2;
        uint32_t pk[kB64 / 2];
        // A row that has seen no key yet (m_used = -inf) has P = 0 by the mask;
        // 0 stands in for its maximum.
        float rs = all ? exp_row<BF, true>(srow, mask, a.scale_log2,
                                           m_used == -INFINITY ? 0.0f : m_used, pk)
                       : exp_row<BF, false>(srow, mask, a.scale_log2,
                                            m_used == -INFINITY ? 0.0f : m_used, pk);
        // The first block set the maximum in use, so its P <= 1.  Later blocks:
        // a row sum above kCheckSum, or a row without a maximum so far, sends
        // the warp to the exact maximum.
        if (!first && __any_sync(0xffffffffu, rs > kCheckSum || m_used == -INFINITY)) {
          const float m_new = row_max_masked(srow, mask) * a.scale_log2;
          const bool need = m_new > m_used + kRescaleLog2;
          if (__any_sync(0xffffffffu, need)) {
            // Recompute P at the new maximum (S is intact: P has not been
            // stored) and rescale O, once the previous P V is done, and l.
            // From -inf the factor is 0, on sums that are 0.
            const float alpha = need ? ex2_approx(m_used - m_new) : 1.0f;
            if (need) m_used = m_new;
            rs = exp_row<BF, false>(srow, mask, a.scale_log2,
                                    m_used == -INFINITY ? 0.0f : m_used, pk);
            if (!(ok = last == b ? true : wait_o(last))) break;
#pragma unroll 1
            for (int c = 0; c < DH; c += 32) {
              float o[32];
              tmem_ld32(orow_t + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              tmem_st32(orow_t + c, o);
            }
            l_run *= alpha;
          }
        }
        l_run += rs;
#pragma unroll
        for (int c = 0; c < kB64 / 2; c += 16) {
          uint32_t q16[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) q16[i] = pk[c + i];
          tmem_st16(srow + c, q16);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
        last = b;
        ++cnt;
      }
      if (ok && total > 0) ok = wait_o(last);
      if (!ok) break;
      g0 += static_cast<uint32_t>(bl.n);
      const bool some = l_run != 0.0f;  // also when it is NaN, and O then is
      const float inv = some ? 1.0f / l_run : 0.0f;
#pragma unroll 1
      for (int h = 0; h < DH / 64; ++h) {
        if (lane == 0) bulk_wait_read<0>();  // the box's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          float v[32];
          if (total > 0) tmem_ld32(orow_t + 64 * h + c, v);
          if (!some) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(box + lane * 128 + (((c / 8 + q) ^ (lane & 7)) << 4)) =
                pack8t<BF>(v + 8 * q, inv);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < a.sq) {
          tma_store_3d(&tmO, box, it.head * DH + 64 * h, row0, it.bi);
          bulk_commit();
        }
      }
      if (r < a.sq)
        a.lse[(static_cast<long long>(it.bi) * a.heads + it.head) * a.sq + r] =
            some ? (m_used + log2f(l_run)) * kLn2 : -INFINITY;
    }
    if (lane == 0) bulk_wait_read<0>();
  }

  __syncwarp();
  tc_fence_before();
  leave(!ok);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ backward

// Row terms of the backward: nd = -rowsum(dO * O), nlse = -LSE * log2(e); a
// row that saw no key (LSE = -inf) gets nlse = -inf, i.e. P = 0.  DH / 8
// threads per (row, head) with 16-byte loads, two pairs in flight.  HBM-bound,
// 4 bytes read per element: 24 us at b = 2, s = 4096, 32 heads of 128 (134
// MB); with 64-bit divisions for the indices the same loop took 36 us.  Blocks
// past the rows zero the row padding and the 64-float tail.
template <bool BF, int DH>
__global__ void __launch_bounds__(256)
    window_dsum(const void* o, long long ldo, const void* d_o, long long lddo, const float* lse,
                float* nlse, float* nd, unsigned pairs, unsigned blocks, unsigned bh, int sq,
                unsigned heads, int sp) {
  constexpr int kLanes = DH / 8, kGroups = 256 / kLanes;
  pdl_next();
  if (blockIdx.x >= blocks) {
    const int padr = sp - sq;
    const long long t = static_cast<long long>(blockIdx.x - blocks) * 256 + threadIdx.x;
    const long long n = static_cast<long long>(bh) * padr;
    if (t < n + 64) {
      const long long i =
          t < n ? t / padr * sp + sq + t % padr : static_cast<long long>(bh) * sp + (t - n);
      nd[i] = 0.0f;
      nlse[i] = 0.0f;
    }
    return;
  }
  const int l = threadIdx.x & (kLanes - 1);
  uint4 ov[2], dv[2];
  float ls[2];
  long long dst[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const unsigned pair = (blockIdx.x * 2 + k) * kGroups + threadIdx.x / kLanes;  // head fastest
    ov[k] = dv[k] = make_uint4(0u, 0u, 0u, 0u);
    ls[k] = 0.0f;
    dst[k] = -1;
    if (pair < pairs) {
      const unsigned row = pair / heads, head = pair - row * heads;
      const unsigned bi = row / static_cast<unsigned>(sq), r = row - bi * sq;
      const long long q = static_cast<long long>(bi) * heads + head;
      ov[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(o) + row * ldo +
                                              head * DH + l * 8);
      dv[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(d_o) + row * lddo +
                                              head * DH + l * 8);
      if (l == 0) ls[k] = lse[q * sq + r];
      dst[k] = q * sp + r;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t ow[4] = {ov[k].x, ov[k].y, ov[k].z, ov[k].w};
    const uint32_t dw[4] = {dv[k].x, dv[k].y, dv[k].z, dv[k].w};
    float acc = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<BF>(ow[i]), y = unpack2<BF>(dw[i]);
      acc = fmaf(x.x, y.x, acc);
      acc = fmaf(x.y, y.y, acc);
    }
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if (l == 0 && dst[k] >= 0) {
      nd[dst[k]] = -acc;
      nlse[dst[k]] = ls[k] == -INFINITY ? -INFINITY : -(ls[k] * kLog2e);
    }
  }
}

constexpr int kKvStages = 3;

template <int DH>
struct DqSmem {
  static constexpr int kTile = 128 * DH * 2, kTile64 = 64 * DH * 2;
  // Q[2] | dO[2] | ring of (K, V) | barriers
  static constexpr int kBytes = 1024 + 4 * kTile + kKvStages * 2 * kTile64 + 256;
};

// dQ: one CTA per (sequence, head, pair of query tiles), 64-key blocks; `cta`
// counts them, heads fastest, longest rows first.  Per block and tile: S = Q
// K^T, dP = dO V^T -> dS over S -> dQ += dS K.  The tensor pipe takes 1024
// clocks of a tile's block (S and dP, operands from shared memory, 768; dQ 256),
// and one warp issues both tiles' products in turn: an issuer per tile, as in
// the forward, was slower (767 against 747 us on the case below).
template <bool BF, int DH>
__device__ __forceinline__ void bwd_dq(const CUtensorMap& tmQ, const CUtensorMap& tmdO,
                                       const CUtensorMap& tmK, const CUtensorMap& tmV, int cta,
                                       const WinArgs& a) {
  constexpr int kTile = DqSmem<DH>::kTile, kTile64 = DqSmem<DH>::kTile64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;               // [2] tiles
  uint8_t* sdO = smem + 2 * kTile;  // [2] tiles
  uint8_t* sKV = smem + 4 * kTile;  // stage st: K at +0, V at +kTile64
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kKvStages * (2 * kTile64));
  uint64_t* qd_full = bars + 0;
  uint64_t* kv_full = bars + 1;              // [kKvStages]
  uint64_t* kv_empty = kv_full + kKvStages;  // [kKvStages]
  uint64_t* s_full = kv_empty + kKvStages;   // [2] tiles: S, dP ready
  uint64_t* ds_full = s_full + 2;            // [2] tiles: dS stored
  uint64_t* dq_done = ds_full + 2;           // [2] tiles
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dq_done + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int npairs = ((a.sq + kBM - 1) / kBM + 1) / 2;
  const int bh = a.bkv * a.group;
  const int pair = npairs - 1 - cta / bh;
  const int head = cta % bh % a.heads, bi = cta % bh / a.heads;
  const int kvh = head / a.group;
  const int r0 = 2 * pair * kBM;
  const BlockList<kB64> bl(r0, a);
  const bool two_terms = split_all(a) || r0 + 2 * kBM + a.off <= kSplitKeys;

  if (threadIdx.x == 0) {
    mbar_init(qd_full, 1);
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&ds_full[i], 4);  // the tile's four element-wise warps
      mbar_init(&dq_done[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, *tmem_slot);  // uniform
  pdl_next();
  pdl_wait();  // the row terms
  // Tile x: S_x at [256 x, +64) (dS_x over its first 32 columns), dP_x at
  // [256 x + 64, +64) (the rest of dS_x over its first 32 columns, if taken),
  // dQ_x at [256 x + 128, + DH).
  auto tS = [tmem](int x) { return tmem + static_cast<uint32_t>(256 * x); };
  auto tP = [tmem](int x) { return tmem + static_cast<uint32_t>(256 * x + 64); };
  auto tQ = [tmem](int x) { return tmem + static_cast<uint32_t>(256 * x + 128); };
  bool ok = true;  // no wait of this thread has given up

  if (warp == 0) {
    if (lane == 0 && bl.n > 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmdO);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      const int tiles = r0 + kBM < a.sq ? 2 : 1;
      mbar_arrive_expect_tx(qd_full, tiles * 2 * kTile);
      for (int x = 0; x < tiles; ++x) {
        load_tile<DH>(sQ + x * kTile, &tmQ, qd_full, head, r0 + x * kBM, bi, 128);
        load_tile<DH>(sdO + x * kTile, &tmdO, qd_full, head, r0 + x * kBM, bi, 128);
      }
      for (int j = 0; j < bl.n && ok; ++j) {
        const int ks = j % kKvStages;
        const uint32_t kph = static_cast<uint32_t>(j / kKvStages) & 1u;
        if (!(ok = mbar_wait(&kv_empty[ks], kph ^ 1u, a.status, kStatusAttnTimeout))) break;
        mbar_arrive_expect_tx(&kv_full[ks], 2 * kTile64);
        uint8_t* dst = sKV + ks * (2 * kTile64);
        const int krow = bl.block(j) * kB64;
        load_tile<DH>(dst, &tmK, &kv_full[ks], kvh, krow, bi, 64);
        load_tile<DH>(dst + kTile64, &tmV, &kv_full[ks], kvh, krow, bi, 64);
      }
    }
  } else if (warp == 1) {
    if (bl.n > 0) {
      constexpr uint32_t kIdSP = idesc<BF>(128, 64, false, false);  // Q K^T, dO V^T
      constexpr uint32_t kIdQ = idesc<BF>(128, DH, false, true);    // dS K
      auto issue_sp = [&](int x, int j) {
        const uint32_t q_addr = smem_u32(sQ + x * kTile), do_addr = smem_u32(sdO + x * kTile);
        const uint32_t k_addr = smem_u32(sKV + (j % kKvStages) * (2 * kTile64));
        const uint32_t v_addr = k_addr + kTile64;
#pragma unroll
        for (int c = 0; c < DH / 64; ++c) {
          warp_umma_ss4(tS(x), sw128_desc(q_addr + c * kBM * 128, 16, 1024),
                        sw128_desc(k_addr + c * kB64 * 128, 16, 1024), kIdSP, c > 0 ? 1u : 0u);
          warp_umma_ss4(tP(x), sw128_desc(do_addr + c * kBM * 128, 16, 1024),
                        sw128_desc(v_addr + c * kB64 * 128, 16, 1024), kIdSP, c > 0 ? 1u : 0u);
        }
        warp_umma_commit(&s_full[x]);
      };
      const int total[2] = {bl.count(0), bl.count(1)};
      int done[2] = {0, 0};
      ok = warp_mbar_wait(qd_full, 0, a.status, kStatusAttnTimeout);
      auto issue = [&](auto two) {
        for (int j = -1; j < bl.n && ok; ++j) {
          const bool more = j + 1 < bl.n;
          bool kv_next = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok) break;
            if (j >= 0 && bl.sees(x, j)) {
              if (!(ok = warp_mbar_wait(&ds_full[x], static_cast<uint32_t>(done[x]) & 1u,
                                        a.status, kStatusAttnTimeout)))
                break;
              tc_fence_after();
              const uint32_t k_addr = smem_u32(sKV + (j % kKvStages) * (2 * kTile64));
              const uint64_t kd = sw128_desc(k_addr, 64 * 128, 1024);
              warp_umma_ts4(tQ(x), tS(x), kd, kIdQ, done[x] > 0 ? 1u : 0u);
              if constexpr (two) warp_umma_ts4(tQ(x), tP(x), kd, kIdQ, 1u);
              if (++done[x] == total[x]) warp_umma_commit(&dq_done[x]);
            }
            if (more && bl.sees(x, j + 1)) {
              if (!kv_next) {
                const int ks = (j + 1) % kKvStages;
                if (!(ok = warp_mbar_wait(&kv_full[ks],
                                          static_cast<uint32_t>((j + 1) / kKvStages) & 1u,
                                          a.status, kStatusAttnTimeout)))
                  break;
                tc_fence_after();
                kv_next = true;
              }
              issue_sp(x, j + 1);
            }
          }
          if (!ok) break;
          if (j >= 0) warp_umma_commit(&kv_empty[j % kKvStages]);
        }
      };
      if (two_terms)
        issue(std::true_type{});
      else
        issue(std::false_type{});
    }
  } else if (warp >= 4) {
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = r0 + x * kBM + quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const long long stat = (static_cast<long long>(bi) * a.heads + head) * a.sp;
    const int rc = min(r, a.sq - 1);
    const float nl = a.nlse[stat + rc], ndd = a.nd[stat + rc];
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(ndd, ndd);
    const int p = rc + a.off;
    const int total = bl.count(x);
    // One loop for tiles that give dS in two terms, one for the others.
    auto blocks = [&](auto two) {
      int cnt = 0;
      for (int j = 0; j < bl.n && cnt < total; ++j) {
        if (!bl.sees(x, j)) continue;
        if (!(ok = mbar_wait(&s_full[x], static_cast<uint32_t>(cnt) & 1u, a.status,
                             kStatusAttnTimeout)))
          break;
        tc_fence_after();
        const RowMask mask = row_mask(p, bl.block(j) * kB64, a);
#pragma unroll
        for (int c = 0; c < kB64; c += 32) {
          float sv[32], pv[32];
          tmem_ld32x2(tS(x) + lane_off + c, sv, tP(x) + lane_off + c, pv);
          uint32_t pk[16];
          const uint32_t vis = mask.full(c) ? 0xffffffffu : mask.bits(c);
          // dS = P (dP - D), two entries at a time; no work for a chunk that no
          // row of the warp sees.
          if (!__any_sync(0xffffffffu, vis != 0u)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0u;
            if constexpr (two) tmem_st16(tP(x) + lane_off + c / 2, pk);
          } else if constexpr (two) {
            uint32_t lk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 t = __ffma2_rn(make_float2(sv[i], sv[i + 1]), sc2, nl2);
              const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
              float2 g = __fmul2_rn(e, __fadd2_rn(make_float2(pv[i], pv[i + 1]), nd2));
              g = make_float2((vis >> i) & 1u ? g.x : 0.0f, (vis >> (i + 1)) & 1u ? g.y : 0.0f);
              split2<BF>(g, pk[i >> 1], lk[i >> 1]);
            }
            tmem_st16(tP(x) + lane_off + c / 2, lk);
          } else if (__all_sync(0xffffffffu, vis == 0xffffffffu)) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 t = __ffma2_rn(make_float2(sv[i], sv[i + 1]), sc2, nl2);
              const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
              const float2 g = __fmul2_rn(e, __fadd2_rn(make_float2(pv[i], pv[i + 1]), nd2));
              pk[i >> 1] = pack2<BF>(g.x, g.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 t = __ffma2_rn(make_float2(sv[i], sv[i + 1]), sc2, nl2);
              const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
              float2 g = __fmul2_rn(e, __fadd2_rn(make_float2(pv[i], pv[i + 1]), nd2));
              g = make_float2((vis >> i) & 1u ? g.x : 0.0f, (vis >> (i + 1)) & 1u ? g.y : 0.0f);
              pk[i >> 1] = pack2<BF>(g.x, g.y);
            }
          }
          // dS columns [c / 2, c / 2 + 16): columns this thread has read.
          tmem_st16(tS(x) + lane_off + c / 2, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[x]);
        ++cnt;
      }
    };
    if (two_terms)
      blocks(std::true_type{});
    else
      blocks(std::false_type{});
    if (ok && total > 0) ok = mbar_wait(&dq_done[x], 0, a.status, kStatusAttnTimeout);
    if (ok) {
      if (total > 0) tc_fence_after();
      uint8_t* out = static_cast<uint8_t*>(a.dq) +
                     ((static_cast<long long>(bi) * a.sq + r) * a.lddq + head * DH) * 2;
#pragma unroll 1
      for (int cc = 0; cc < DH; cc += 32) {
        float v[32];
        if (total > 0) {
          tmem_ld32(tQ(x) + lane_off + cc, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        }
        if (r < a.sq) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(out + 2 * (cc + 8 * q)) = pack8t<BF>(v + 8 * q, a.scale);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  leave(!ok);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

constexpr int kQdStages = 4;

template <int DH>
struct KvSmem {
  static constexpr int kTile = 128 * DH * 2, kTile64 = 64 * DH * 2;
  // K | V | ring of (Q, dO) | barriers | ring of row terms (128 floats)
  static constexpr int kBytes =
      1024 + 2 * kTile + kQdStages * 2 * kTile64 + 256 + kQdStages * 2 * kB64 * 4;
};

// Query blocks of 64 that see some key of the tile at k0: [i0, i0 + n).
struct QRange {
  int i0, n;
};

__host__ __device__ __forceinline__ QRange query_blocks(int k0, int sq, int sk, int window,
                                                        int sinks) {
  const int off = sk - sq;
  const int k1 = (k0 + kBN < sk ? k0 + kBN : sk) - 1;
  const int lo = k0 - off > 0 ? k0 - off : 0;
  int hi = sq - 1;
  if (k0 >= sinks) {
    const long long w = static_cast<long long>(k1) + window - 1 - off;
    if (w < hi) hi = static_cast<int>(w);
  }
  QRange q;
  q.i0 = lo / kB64;
  q.n = lo <= hi ? hi / kB64 - q.i0 + 1 : 0;
  return q;
}

// Work item k of the dK / dV kernel: a slice [j0, j1) of the (head, query
// block) list of one (sequence, key head, key tile); list entry j is query
// block i0 + j % n of head kvh * group + j / n.  The sink tiles' slices come
// first (they are the longest).
struct KvItem {
  int bi, kvh, k0, i0, n, j0, j1;
  int slot;  // slice of the partials, -1: the tile is not cut
  bool two;  // P and dS in two terms
};

__device__ __forceinline__ KvItem kv_item(int k, const WinArgs& a) {
  KvItem it;
  const int sink_items = a.sink_tiles * a.split_s * a.bkv;
  int split, s, kb, bk;
  if (k < sink_items) {
    split = a.split_s;
    bk = k % a.bkv;
    const int v = k / a.bkv;
    s = v % split;
    kb = v / split;
    it.slot = split > 1 ? (kb * a.bkv + bk) * split + s : -1;
  } else {
    const int v0 = k - sink_items;
    split = a.split_w;
    bk = v0 % a.bkv;
    const int v = v0 / a.bkv;
    s = v % split;
    kb = v / split;  // among the tiles without sinks
    it.slot = split > 1 ? (a.split_s > 1 ? sink_items : 0) + (kb * a.bkv + bk) * split + s : -1;
    kb += a.sink_tiles;
  }
  it.kvh = bk % a.kv_heads;
  it.bi = bk / a.kv_heads;
  it.k0 = kb * kBN;
  it.two = split_all(a) || it.k0 < kSplitKeys;
  const QRange q = query_blocks(it.k0, a.sq, a.sk, a.window, a.sinks);
  it.i0 = q.i0;
  it.n = q.n;
  const long long len = static_cast<long long>(q.n) * a.group;
  it.j0 = static_cast<int>(s * len / split);
  it.j1 = static_cast<int>((s + 1) * len / split);
  return it;
}

// The r-th item of this CTA, or -1: rounds of kv_ctas items in snake order.
__device__ __forceinline__ int kv_item_index(int r, const WinArgs& a) {
  const long long g = a.kv_ctas, c = blockIdx.x;
  const long long k = r * g + ((r & 1) ? g - 1 - c : c);
  return k < a.items ? static_cast<int>(k) : -1;
}

// Persistent dK / dV: one CTA per SM walks its items; per 64-query block
// S^T = K Q^T, dP^T = V dO^T -> P^T, dS^T -> dV += P^T dO, dK += dS^T Q.
// The Q / dO ring runs on across items; an item's K and V load once the
// previous item's last S^T / dP^T are done (kv_empty), and its first dV, dK
// products wait until the previous epilogue has read the accumulators
// (acc_empty).  Items without queries only write zeros.
// The tensor pipe takes 1280 clocks of a block of 64 queries, a block about 2200: the
// element-wise warps take about 1500 of them from S^T to P^T.  Both parts on two
// sequences of 4096, 32 + 8 heads of 128, window 1024, 4 sinks (301 GFLOP): 520
// us at 1.69 GHz, 579 TFLOP/s; with the products issued under a branch to one
// lane 630-676 us.
template <bool BF, int DH>
__device__ __forceinline__ void bwd_dkdv(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                         const CUtensorMap& tmQ, const CUtensorMap& tmdO,
                                         const WinArgs& a) {
  constexpr int kTile = KvSmem<DH>::kTile, kTile64 = KvSmem<DH>::kTile64;
  constexpr int kEwWarps = 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + kTile;
  uint8_t* sQdO = smem + 2 * kTile;  // stage q: Q at +0, dO at +kTile64
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQdO + kQdStages * (2 * kTile64));
  uint64_t* kv_full = bars + 0;
  uint64_t* kv_empty = bars + 1;             // the item's last S^T / dP^T done
  uint64_t* qd_full = bars + 2;              // [kQdStages]
  uint64_t* qd_empty = qd_full + kQdStages;  // [kQdStages]
  uint64_t* s_full = qd_empty + kQdStages;   // [2]
  uint64_t* p_full = s_full + 2;             // [2]
  uint64_t* acc_done = p_full + 2;           // the item's last dV, dK products done
  uint64_t* acc_empty = acc_done + 1;        // the epilogue has read dV, dK
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
  // stage q: -LSE * log2(e) of the block's 64 queries at [0, 64), -D at [64, 128)
  float* s_stat = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (int i = 0; i < kQdStages; ++i) {
      mbar_init(&qd_full[i], 1);
      mbar_init(&qd_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kEwWarps);
    }
    mbar_init(acc_done, 1);
    mbar_init(acc_empty, kEwWarps);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, *tmem_slot);  // uniform
  pdl_next();
  pdl_wait();  // the row terms
  // S^T buffers at columns 0 and 64, dP^T at 128 and 192, dV at 256, dK at 384.
  auto tS = [tmem](int st) { return tmem + static_cast<uint32_t>(64 * st); };
  auto tP = [tmem](int st) { return tmem + static_cast<uint32_t>(128 + 64 * st); };
  const uint32_t tdV = tmem + 256, tdK = tmem + 384;
  bool ok = true;  // no wait of this thread has given up

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmdO);
      long long g = 0;  // query blocks loaded so far: the ring position
      uint32_t it_no = 0;  // items with queries so far
      for (int r = 0; ok; ++r) {
        const int k = kv_item_index(r, a);
        if (k < 0) break;
        const KvItem it = kv_item(k, a);
        if (it.j0 >= it.j1) continue;
        if (!(ok = mbar_wait(kv_empty, (it_no & 1u) ^ 1u, a.status, kStatusAttnTimeout))) break;
        ++it_no;
        mbar_arrive_expect_tx(kv_full, 2 * kTile);
        load_tile<DH>(sK, &tmK, kv_full, it.kvh, it.k0, it.bi, 128);
        load_tile<DH>(sV, &tmV, kv_full, it.kvh, it.k0, it.bi, 128);
        int hg = it.j0 / it.n, qi = it.j0 - hg * it.n;
        for (int j = it.j0; j < it.j1; ++j, ++g) {
          const int qs = static_cast<int>(g % kQdStages);
          const uint32_t qph = static_cast<uint32_t>(g / kQdStages) & 1u;
          if (!(ok = mbar_wait(&qd_empty[qs], qph ^ 1u, a.status, kStatusAttnTimeout))) break;
          const int q0 = (it.i0 + qi) * kB64;
          const int head = it.kvh * a.group + hg;
          mbar_arrive_expect_tx(&qd_full[qs], 2 * kTile64 + 2 * kB64 * 4);
          uint8_t* dst = sQdO + qs * (2 * kTile64);
          load_tile<DH>(dst, &tmQ, &qd_full[qs], head, q0, it.bi, 64);
          load_tile<DH>(dst + kTile64, &tmdO, &qd_full[qs], head, q0, it.bi, 64);
          // The block's row terms; past sq they are zeros or the next row's
          // values, which the mask never lets through.
          const long long stat = (static_cast<long long>(it.bi) * a.heads + head) * a.sp + q0;
          float* st_dst = s_stat + qs * (2 * kB64);
          bulk_load(st_dst, a.nlse + stat, kB64 * 4, &qd_full[qs]);
          bulk_load(st_dst + kB64, a.nd + stat, kB64 * 4, &qd_full[qs]);
          if (++qi == it.n) {
            qi = 0;
            ++hg;
          }
        }
      }
    }
  } else if (warp == 1) {
    {
      constexpr uint32_t kIdSP = idesc<BF>(128, 64, false, false);  // K Q^T, V dO^T
      constexpr uint32_t kIdAcc = idesc<BF>(128, DH, false, true);  // P^T dO, dS^T Q
      const uint32_t k_addr = smem_u32(sK), v_addr = smem_u32(sV);
      // S^T / dP^T of ring position gg into buffer gg & 1, whose P^T / dS^T
      // the products of position gg - 2 (issued before) have read.
      auto issue_sp = [&](long long gg) -> bool {
        const int st = static_cast<int>(gg & 1);
        const int qs = static_cast<int>(gg % kQdStages);
        if (!warp_mbar_wait(&qd_full[qs], static_cast<uint32_t>(gg / kQdStages) & 1u, a.status,
                       kStatusAttnTimeout))
          return false;
        tc_fence_after();
        const uint32_t q_addr = smem_u32(sQdO + qs * (2 * kTile64));
        const uint32_t do_addr = q_addr + kTile64;
#pragma unroll
        for (int c = 0; c < DH / 64; ++c) {
          warp_umma_ss4(tS(st), sw128_desc(k_addr + c * kBN * 128, 16, 1024),
                        sw128_desc(q_addr + c * kB64 * 128, 16, 1024), kIdSP, c > 0 ? 1u : 0u);
          warp_umma_ss4(tP(st), sw128_desc(v_addr + c * kBN * 128, 16, 1024),
                        sw128_desc(do_addr + c * kB64 * 128, 16, 1024), kIdSP, c > 0 ? 1u : 0u);
        }
        warp_umma_commit(&s_full[st]);
        return true;
      };
      long long g = 0;  // query blocks of the items before this one
      uint32_t it_no = 0;
      for (int r = 0; ok; ++r) {
        const int k = kv_item_index(r, a);
        if (k < 0) break;
        const KvItem it = kv_item(k, a);
        const int len = it.j1 - it.j0;
        if (len <= 0) continue;
        if (!(ok = warp_mbar_wait(kv_full, it_no & 1u, a.status, kStatusAttnTimeout))) break;
        if (!(ok = issue_sp(g))) break;
        if (len == 1) warp_umma_commit(kv_empty);
        auto issue = [&](auto two) {
          for (int j = 0; j < len; ++j) {
            const long long gj = g + j;
            if (j + 1 < len) {
              if (!(ok = issue_sp(gj + 1))) break;
              if (j + 2 == len) warp_umma_commit(kv_empty);  // the item's last S^T / dP^T
            }
            const int st = static_cast<int>(gj & 1);
            if (!(ok = warp_mbar_wait(&p_full[st], static_cast<uint32_t>(gj >> 1) & 1u, a.status,
                                 kStatusAttnTimeout)))
              break;
            // The item's first products overwrite the accumulators: the previous
            // item's epilogue must have read them.
            if (j == 0 && it_no > 0 &&
                !(ok = warp_mbar_wait(acc_empty, (it_no - 1u) & 1u, a.status, kStatusAttnTimeout)))
              break;
            tc_fence_after();
            const int qs = static_cast<int>(gj % kQdStages);
            const uint32_t q_addr = smem_u32(sQdO + qs * (2 * kTile64));
            const uint32_t do_addr = q_addr + kTile64;
            // 32 queries lie 32 columns apart, their second terms 16 columns on
            const uint64_t dod = sw128_desc(do_addr, 64 * 128, 1024);
            const uint64_t qd = sw128_desc(q_addr, 64 * 128, 1024);
            warp_umma_ts4<32>(tdV, tS(st), dod, kIdAcc, j > 0 ? 1u : 0u);
            warp_umma_ts4<32>(tdK, tP(st), qd, kIdAcc, j > 0 ? 1u : 0u);
            if constexpr (two) {
              warp_umma_ts4<32>(tdV, tS(st) + 16, dod, kIdAcc, 1u);
              warp_umma_ts4<32>(tdK, tP(st) + 16, qd, kIdAcc, 1u);
            }
            warp_umma_commit(&qd_empty[qs]);
          }
        };
        if (it.two)
          issue(std::true_type{});
        else
          issue(std::false_type{});
        if (!ok) break;
        warp_umma_commit(acc_done);
        g += len;
        ++it_no;
      }
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    const int grp = (warp - 4) >> 2;  // this warp's column half
    const int c = grp * 32;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    long long gb = 0;  // query blocks of the items before this one
    uint32_t it_no = 0;
    for (int ri = 0; ok; ++ri) {
      const int k = kv_item_index(ri, a);
      if (k < 0) break;
      const KvItem it = kv_item(k, a);
      const int key = it.k0 + r;
      const int len = it.j1 - it.j0;
      // queries [qlo, qhi) see this key
      const int qlo = key - a.off;
      int qhi = a.sq;
      if (key >= a.sinks)
        qhi = static_cast<int>(min(static_cast<long long>(a.sq),
                                   static_cast<long long>(key) + a.window - a.off));
      if (key >= a.sk) qhi = 0;
      int qi = it.n > 0 ? it.j0 % it.n : 0;
      auto blocks = [&](auto two) {
        for (int j = 0; j < len; ++j) {
          const long long gj = gb + j;
          const int st = static_cast<int>(gj & 1);
          const int qs = static_cast<int>(gj % kQdStages);
          const int q0 = (it.i0 + qi) * kB64;
          if (++qi == it.n) qi = 0;
          // The block's row terms were staged with its Q / dO; the stage cannot
          // be refilled before this block's products are done.  -LSE is read
          // before S is there: while products run they take all of shared
          // memory's bandwidth (896k cycles for the launch on the case above,
          // 918k without; -D as well would spill, 909k).
          if (!(ok = mbar_wait(&qd_full[qs], static_cast<uint32_t>(gj / kQdStages) & 1u, a.status,
                               kStatusAttnTimeout)))
            break;
          const float4* wnl = reinterpret_cast<const float4*>(s_stat + qs * (2 * kB64) + c);
          const float4* wnd = wnl + kB64 / 4;
          float4 nl4[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) nl4[i] = wnl[i];
          if (!(ok = mbar_wait(&s_full[st], static_cast<uint32_t>(gj >> 1) & 1u, a.status,
                               kStatusAttnTimeout)))
            break;
          tc_fence_after();
          const int lo = qlo - q0 - c, hi = qhi - q0 - c;  // visible columns lo <= i < hi
          float sv[32], pv[32];
          tmem_ld32x2(tS(st) + lane_off + c, sv, tP(st) + lane_off + c, pv);
          uint32_t pk[16], dk[16];
          const bool full = lo <= 0 && hi >= 32;
          const uint32_t vis = full ? 0xffffffffu : RowMask::prefix(hi) & ~RowMask::prefix(lo);
          if (!__any_sync(0xffffffffu, vis != 0u)) {  // no key of this warp sees a query
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = dk[i] = 0u;
            if constexpr (two) {
              tmem_st16(tS(st) + lane_off + c + 16, pk);
              tmem_st16(tP(st) + lane_off + c + 16, dk);
            }
          } else if constexpr (two) {
            uint32_t pl[16], dl[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 nl = half4(nl4[i >> 2], i), nd = half4(wnd[i >> 2], i);
              const float2 t = __ffma2_rn(make_float2(sv[i], sv[i + 1]), sc2, nl);
              float2 d = __fadd2_rn(make_float2(pv[i], pv[i + 1]), nd);
              const bool v0 = (vis >> i) & 1u, v1 = (vis >> (i + 1)) & 1u;
              const float2 p =
                make_float2(v0 ? ex2_approx(t.x) : 0.0f, v1 ? ex2_approx(t.y) : 0.0f);
              d = make_float2(v0 ? d.x : 0.0f, v1 ? d.y : 0.0f);
              split2<BF>(p, pk[i >> 1], pl[i >> 1]);
              split2<BF>(__fmul2_rn(p, d), dk[i >> 1], dl[i >> 1]);
            }
            tmem_st16(tS(st) + lane_off + c + 16, pl);
            tmem_st16(tP(st) + lane_off + c + 16, dl);
          } else if (__all_sync(0xffffffffu, full)) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 nl = half4(nl4[i >> 2], i), nd = half4(wnd[i >> 2], i);
              const float2 t = __ffma2_rn(make_float2(sv[i], sv[i + 1]), sc2, nl);
              const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
              const float2 g = __fmul2_rn(p, __fadd2_rn(make_float2(pv[i], pv[i + 1]), nd));
              pk[i >> 1] = pack2<BF>(p.x, p.y);
              dk[i >> 1] = pack2<BF>(g.x, g.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 nl = half4(nl4[i >> 2], i), nd = half4(wnd[i >> 2], i);
              const float2 t = __ffma2_rn(make_float2(sv[i], sv[i + 1]), sc2, nl);
              float2 d = __fadd2_rn(make_float2(pv[i], pv[i + 1]), nd);
              // hidden queries may stand on the row terms of another sequence
              const bool v0 = (vis >> i) & 1u, v1 = (vis >> (i + 1)) & 1u;
              const float2 p =
                  make_float2(v0 ? ex2_approx(t.x) : 0.0f, v1 ? ex2_approx(t.y) : 0.0f);
              d = make_float2(v0 ? d.x : 0.0f, v1 ? d.y : 0.0f);
              const float2 g = __fmul2_rn(p, d);
              pk[i >> 1] = pack2<BF>(p.x, p.y);
              dk[i >> 1] = pack2<BF>(g.x, g.y);
            }
          }
          tmem_st16(tS(st) + lane_off + c, pk);  // P^T over this group's S^T columns
          tmem_st16(tP(st) + lane_off + c, dk);  // dS^T over its dP^T columns
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[st]);
        }
      };
      if (it.two)
        blocks(std::true_type{});
      else
        blocks(std::false_type{});
      if (!ok) break;
      if (len > 0) {
        gb += len;
        if (!(ok = mbar_wait(acc_done, it_no & 1u, a.status, kStatusAttnTimeout))) break;
        ++it_no;
        tc_fence_after();
      }
      const long long row = static_cast<long long>(it.bi) * a.sk + key;
      uint8_t* okp = static_cast<uint8_t*>(a.dk) + (row * a.lddk + it.kvh * DH) * 2;
      uint8_t* ovp = static_cast<uint8_t*>(a.dv) + (row * a.lddv + it.kvh * DH) * 2;
      // partials: [slot][dK, dV][DH / 4][128 keys][4], so a warp's 32 rows
      // store 512 contiguous bytes
      float4* part = reinterpret_cast<float4*>(a.part) +
                     static_cast<long long>(max(it.slot, 0)) * 2 * 128 * (DH / 4);
#pragma unroll
      for (int cc = grp * (DH / 2); cc < (grp + 1) * (DH / 2); cc += 32) {
        float vk[32], vv[32];
        if (len > 0) {
          tmem_ld32(tdK + lane_off + cc, vk);
          tmem_ld32(tdV + lane_off + cc, vv);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) vk[i] = vv[i] = 0.0f;
        }
        if (it.slot >= 0) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            part[(cc / 4 + q) * 128 + r] =
                make_float4(vk[4 * q], vk[4 * q + 1], vk[4 * q + 2], vk[4 * q + 3]);
            part[128 * (DH / 4) + (cc / 4 + q) * 128 + r] =
                make_float4(vv[4 * q], vv[4 * q + 1], vv[4 * q + 2], vv[4 * q + 3]);
          }
        } else if (key < a.sk) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            *reinterpret_cast<uint4*>(okp + 2 * (cc + 8 * q)) = pack8t<BF>(vk + 8 * q, a.scale);
            *reinterpret_cast<uint4*>(ovp + 2 * (cc + 8 * q)) = pack8t<BF>(vv + 8 * q, 1.0f);
          }
        }
      }
      if (len > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  leave(!ok);
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Both in one launch: the persistent dK / dV CTAs first, then the dQ CTAs,
// which fill the SMs that the static split of the key tiles leaves idle at its
// end (and, on small problems, run beside them).
template <bool BF, int DH>
__global__ void __launch_bounds__(kThreads, 1)
    window_bwd(const __grid_constant__ CUtensorMap q128, const __grid_constant__ CUtensorMap do128,
               const __grid_constant__ CUtensorMap k64, const __grid_constant__ CUtensorMap v64,
               const __grid_constant__ CUtensorMap k128, const __grid_constant__ CUtensorMap v128,
               const __grid_constant__ CUtensorMap q64, const __grid_constant__ CUtensorMap do64,
               const WinArgs a) {
  if (static_cast<int>(blockIdx.x) < a.kv_ctas)
    bwd_dkdv<BF, DH>(k128, v128, q64, do64, a);
  else
    bwd_dq<BF, DH>(q128, do128, k64, v64, static_cast<int>(blockIdx.x) - a.kv_ctas, a);
}

// Adds the slices of one cut key tile in slice order and writes dK (scaled)
// and dV.  Block (tile slot group, 8 columns, dK or dV): thread = key row.
template <bool BF, int DH>
__global__ void __launch_bounds__(128) window_kv_join(const WinArgs a, int first_tile, int split,
                                                      int slot0) {
  pdl_next();
  pdl_wait();  // the partials
  const int bk = blockIdx.x % a.bkv, kb = blockIdx.x / a.bkv;  // kb: among the class's tiles
  const int c8 = blockIdx.y, which = blockIdx.z;
  const int kvh = bk % a.kv_heads, bi = bk / a.kv_heads;
  const int key = (first_tile + kb) * kBN + threadIdx.x;
  if (key >= a.sk) return;
  const float4* p = reinterpret_cast<const float4*>(a.part) +
                    (static_cast<long long>(slot0) +
                     static_cast<long long>(kb * a.bkv + bk) * split) *
                        (2 * 128 * (DH / 4)) +
                    which * 128 * (DH / 4) + c8 * 2 * 128 + threadIdx.x;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < split; ++s) {
    const float4 x = __ldcg(p + static_cast<long long>(s) * 2 * 128 * (DH / 4));
    const float4 y = __ldcg(p + static_cast<long long>(s) * 2 * 128 * (DH / 4) + 128);
    v[0] += x.x;
    v[1] += x.y;
    v[2] += x.z;
    v[3] += x.w;
    v[4] += y.x;
    v[5] += y.y;
    v[6] += y.z;
    v[7] += y.w;
  }
  const long long row = static_cast<long long>(bi) * a.sk + key;
  uint8_t* out = which == 0
                     ? static_cast<uint8_t*>(a.dk) + (row * a.lddk + kvh * DH + c8 * 8) * 2
                     : static_cast<uint8_t*>(a.dv) + (row * a.lddv + kvh * DH + c8 * 8) * 2;
  *reinterpret_cast<uint4*>(out) = pack8t<BF>(v, which == 0 ? a.scale : 1.0f);
}

// ------------------------------------------------------------------ host side

// [seqs][rows][cols] two-byte matrix with row stride ld (elements); boxes of
// 64 columns x box_rows rows of one sequence, 128-byte swizzle.
bool make_map3(CUtensorMap* m, const void* ptr, bool bf, int64_t cols, int64_t rows, int64_t seqs,
               int64_t ld, int box_rows) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(seqs)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld * rows) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the key tiles of the dK / dV kernel are cut.  A slice takes about half
// of an SM's share of all blocks, so the items balance, but at least 16 blocks
// (about 1.1 us each; its partials cost 128 KB of traffic), or, where that
// leaves SMs without an item, an SM's share, at least 4.
constexpr int kMaxSlices = 255;

struct KvPlan {
  int key_tiles, sink_tiles, split_s, split_w;
  int64_t items, slots;
};

KvPlan plan_kv(const WindowAttn& w) {
  KvPlan p{};
  p.key_tiles = static_cast<int>((w.sk + kBN - 1) / kBN);
  p.sink_tiles = static_cast<int>((w.sinks + kBN - 1) / kBN);
  const int64_t bkv = w.b * w.kv_heads, group = w.heads / w.kv_heads;
  int64_t blocks = 0, max_s = 0, max_w = 0;
  for (int kb = 0; kb < p.key_tiles; ++kb) {
    const int64_t n = group * query_blocks(kb * kBN, static_cast<int>(w.sq), static_cast<int>(w.sk),
                                           static_cast<int>(w.window), static_cast<int>(w.sinks)).n;
    blocks += n;
    int64_t& mx = kb < p.sink_tiles ? max_s : max_w;
    mx = std::max(mx, n);
  }
  const int64_t share = blocks * bkv / sm_count();
  const int64_t slice =
      std::max<int64_t>({4, std::min<int64_t>(16, share), share / 2});
  auto cut = [&](int64_t n) {
    return static_cast<int>(
        std::min<int64_t>(kMaxSlices, std::max<int64_t>(1, (n + slice - 1) / slice)));
  };
  p.split_s = cut(max_s);
  p.split_w = cut(max_w);
  const int64_t ns = int64_t(p.sink_tiles) * bkv * p.split_s;
  const int64_t nw = int64_t(p.key_tiles - p.sink_tiles) * bkv * p.split_w;
  p.items = ns + nw;
  p.slots = (p.split_s > 1 ? ns : 0) + (p.split_w > 1 ? nw : 0);
  return p;
}

int64_t stat_stride(int64_t s) { return (s + 3) / 4 * 4; }

size_t stat_bytes(const WindowAttn& w) {
  const size_t n = static_cast<size_t>(w.b * w.heads) * stat_stride(w.sq) + 64;
  return (n * sizeof(float) + 255) / 256 * 256;
}

WinArgs base_args(const WindowAttn& w) {
  WinArgs a{};
  a.sq = static_cast<int>(w.sq);
  a.sk = static_cast<int>(w.sk);
  a.off = a.sk - a.sq;
  a.heads = w.heads;
  a.kv_heads = w.kv_heads;
  a.group = w.heads / w.kv_heads;
  a.window = static_cast<int>(w.window);
  a.sinks = static_cast<int>(w.sinks);
  a.scale = w.scale;
  a.scale_log2 = w.scale * kLog2e;
  a.status = wait_ctl();
  return a;
}

// Visible (query, key) pairs of all heads.
double visible_pairs(const WindowAttn& w) {
  double n = 0;
  const double off = double(w.sk - w.sq);
  // rows with p + 1 <= window + sinks see p + 1 keys, later ones window + sinks
  const double p0 = std::max(0.0, off), p1 = double(w.sk);  // positions [p0, p1)
  const double m = std::min(std::max(double(w.window + w.sinks), p0), p1);
  n += (m * (m + 1) - p0 * (p0 + 1)) / 2;
  n += (p1 - m) * double(w.window + w.sinks);
  return n * double(w.b) * w.heads;
}

template <typename K>
tp_status smem_opt_in(K kern, int bytes, const char* what) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e == cudaSuccess ? TP_OK : cuda_fail(e, what);
}

template <bool BF, int DH>
tp_status fwd(const WindowAttn& w, cudaStream_t stream) {
  CUtensorMap q, k, v, o;
  const int64_t nq = int64_t(w.heads) * DH, nk = int64_t(w.kv_heads) * DH;
  if (!make_map3(&q, w.q, BF, nq, w.sq, w.b, w.ldq, 128) ||
      !make_map3(&k, w.k, BF, nk, w.sk, w.b, w.ldk, kB64) ||
      !make_map3(&v, w.v, BF, nk, w.sk, w.b, w.ldv, kB64) ||
      !make_map3(&o, w.o, BF, nq, w.sq, w.b, w.ldo, 32))
    return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled failed (window attention)");
  WinArgs a = base_args(w);
  if (a.status.st == nullptr) return fail(TP_ERR_CUDA, "device status unavailable");
  a.lse = const_cast<float*>(w.lse);
  constexpr int smem = FwdSmem<DH>::kBytes;
  if (tp_status s = smem_opt_in(window_fwd<BF, DH>, smem, "window attention smem"); s != TP_OK)
    return s;
  const int64_t npairs = ((w.sq + kBM - 1) / kBM + 1) / 2;
  a.bkv = static_cast<int>(w.b * w.kv_heads);
  a.items = static_cast<int>(npairs * w.b * w.heads);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.items, sm_count()));
  {
    LaunchScope scope(TP_KIND_ATTN_FWD, 4.0 * DH * visible_pairs(w),
                      4.0 * double(w.b) * (w.sq * nq + w.sk * nk), stream);
    window_fwd<BF, DH><<<grid, kThreads, smem, stream>>>(q, k, v, o, a);
  }
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TP_OK : cuda_fail(e, "window attention forward launch");
}

template <bool BF, int DH>
tp_status bwd(const WindowAttn& w, void* scratch, cudaStream_t stream) {
  CUtensorMap q128, do128, k64, v64, k128, v128, q64, do64;
  const int64_t nq = int64_t(w.heads) * DH, nk = int64_t(w.kv_heads) * DH;
  if (!make_map3(&q128, w.q, BF, nq, w.sq, w.b, w.ldq, 128) ||
      !make_map3(&do128, w.d_o, BF, nq, w.sq, w.b, w.lddo, 128) ||
      !make_map3(&k64, w.k, BF, nk, w.sk, w.b, w.ldk, 64) ||
      !make_map3(&v64, w.v, BF, nk, w.sk, w.b, w.ldv, 64) ||
      !make_map3(&k128, w.k, BF, nk, w.sk, w.b, w.ldk, 128) ||
      !make_map3(&v128, w.v, BF, nk, w.sk, w.b, w.ldv, 128) ||
      !make_map3(&q64, w.q, BF, nq, w.sq, w.b, w.ldq, 64) ||
      !make_map3(&do64, w.d_o, BF, nq, w.sq, w.b, w.lddo, 64))
    return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled failed (window attention backward)");
  WinArgs a = base_args(w);
  if (a.status.st == nullptr) return fail(TP_ERR_CUDA, "device status unavailable");
  const size_t sb = stat_bytes(w);
  float* nlse = static_cast<float*>(scratch);
  float* nd = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + sb);
  a.nlse = nlse;
  a.nd = nd;
  a.sp = static_cast<int>(stat_stride(w.sq));
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + 2 * sb);
  a.dq = w.dq;
  a.dk = w.dk;
  a.dv = w.dv;
  a.lddq = w.lddq;
  a.lddk = w.lddk;
  a.lddv = w.lddv;
  const KvPlan p = plan_kv(w);
  a.bkv = static_cast<int>(w.b * w.kv_heads);
  a.key_tiles = p.key_tiles;
  a.sink_tiles = p.sink_tiles;
  a.split_s = p.split_s;
  a.split_w = p.split_w;
  a.items = static_cast<int>(p.items);
  constexpr int smem = std::max(DqSmem<DH>::kBytes, KvSmem<DH>::kBytes);
  if (tp_status s = smem_opt_in(window_bwd<BF, DH>, smem, "window backward smem"); s != TP_OK)
    return s;
  const int64_t rows = w.b * w.sq;
  const int64_t pad = w.b * w.heads * (a.sp - w.sq) + 64;
  const int64_t pairs = rows * w.heads, per_block = 2 * 256 / (DH / 8);
  const int64_t dsum_rows = (pairs + per_block - 1) / per_block;
  const int64_t dsum_blocks = dsum_rows + (pad + 255) / 256;
  const int64_t npairs = ((w.sq + kBM - 1) / kBM + 1) / 2;
  a.kv_ctas = static_cast<int>(std::min<int64_t>(p.items, sm_count()));
  const unsigned grid = static_cast<unsigned>(w.b * w.heads * npairs + a.kv_ctas);
  const int joins = (p.split_s > 1) + (p.split_w > 1 && p.key_tiles > p.sink_tiles);
  LaunchScope scope(TP_KIND_ATTN_BWD, 10.0 * DH * visible_pairs(w),
                    double(w.b) * (8.0 * w.sq * nq + 8.0 * w.sk * nk), stream, 2 + joins);
  window_dsum<BF, DH><<<static_cast<unsigned>(dsum_blocks), 256, 0, stream>>>(
      w.o, w.ldo, w.d_o, w.lddo, w.lse, nlse, nd, static_cast<unsigned>(pairs),
      static_cast<unsigned>(dsum_rows), static_cast<unsigned>(w.b * w.heads), a.sq,
      static_cast<unsigned>(a.heads), a.sp);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_kernel(window_bwd<BF, DH>, dim3(grid), kThreads, smem, stream, true, q128, do128, k64,
                      v64, k128, v128, q64, do64, a);
  if (e == cudaSuccess && p.split_s > 1)
    e = launch_kernel(window_kv_join<BF, DH>, dim3(p.sink_tiles * a.bkv, DH / 8, 2), 128, 0,
                      stream, true, a, 0, p.split_s, 0);
  if (e == cudaSuccess && p.split_w > 1 && p.key_tiles > p.sink_tiles)
    e = launch_kernel(window_kv_join<BF, DH>,
                      dim3((p.key_tiles - p.sink_tiles) * a.bkv, DH / 8, 2), 128, 0, stream, true,
                      a, p.sink_tiles, p.split_w,
                      p.split_s > 1 ? p.sink_tiles * a.bkv * p.split_s : 0);
  return e == cudaSuccess ? TP_OK : cuda_fail(e, "window attention backward launch");
}

}  // namespace

tp_status window_attn_check(const WindowAttn& w) {
  const int64_t q_tiles = (w.sq + kBM - 1) / kBM;
  if (q_tiles > 65535 || w.b * w.heads > 0x10000000LL || w.b * w.heads * q_tiles > 0x70000000LL)
    return fail(TP_ERR_SHAPE, "window attention: sequence or b * heads too large");
  const int64_t tiles = (w.sk + kBN - 1) / kBN;
  if (tiles * w.b * w.kv_heads > 0x7fffffffLL / kMaxSlices ||
      (w.sq + kB64 - 1) / kB64 * (w.heads / w.kv_heads) > 0x7fffffffLL ||
      w.b * w.sq * w.heads > 0xe0000000LL)
    return fail(TP_ERR_SHAPE, "window attention: too many key tiles");
  return TP_OK;
}

size_t window_attn_scratch_bytes(const WindowAttn& w) {
  return 2 * stat_bytes(w) + static_cast<size_t>(plan_kv(w).slots) * 2 * kBN * w.d * 4;
}

tp_status launch_window_attn_fwd(const WindowAttn& w, cudaStream_t stream) {
  if (w.dtype == TP_BF16)
    return w.d == 64 ? fwd<true, 64>(w, stream) : fwd<true, 128>(w, stream);
  return w.d == 64 ? fwd<false, 64>(w, stream) : fwd<false, 128>(w, stream);
}

tp_status launch_window_attn_bwd(const WindowAttn& w, void* scratch, cudaStream_t stream) {
  if (w.dtype == TP_BF16)
    return w.d == 64 ? bwd<true, 64>(w, scratch, stream) : bwd<true, 128>(w, scratch, stream);
  return w.d == 64 ? bwd<false, 64>(w, scratch, stream) : bwd<false, 128>(w, scratch, stream);
}

}  // namespace tp
