// The gated feed-forward block on a few tokens: the cost is reading the
// weights once (2 M flops per weight byte, far below the ridge), so both
// products stream them.
//   up:   H = act(X Wg + bg) * (X Wu + bu)   (gate and up columns together)
//   down: Z = H Wd + bd
// * A block owns 64 columns of H (its gate and its up columns) or 128 of Z and
//   a slice of K; its 8 warps are 4 K groups x 2 runs of 64 columns.  A warp
//   streams its own 16 (K) x 64 (columns) weight tiles, with the tokens' 16
//   values of K beside them, through its own ring of cp.async stages: no block
//   barrier in the loop, 128 contiguous bytes per weight row.
// * m16n8k16 products, 16 tokens as the rows (MT of them per warp), the weight
//   tile transposed on its way out of shared memory.
// * The K groups are added through shared memory, the K slices of a tile
//   (a cluster of blocks) through distributed shared memory, in a fixed
//   order; then bias, activation and product.  Nothing goes through HBM but
//   the weights, X, H and Z.
// * H is rounded to bf16 between the products, as in the larger batches' GEMM,
//   which makes a token's Z 1.4 times as far off as its own rounding.  Up to 8
//   tokens the rounded rest follows as a second term, because it is nearly free
//   there: 60.4 against 59.2 us for one token, 66 for 8 (9 with one term 64).
//   That is a trade of speed alone, a token's accuracy does not gain from
//   company: at 13 tokens the second term would cost 6% (25.1 against 23.6 us),
//   at 32 tokens 12%, in the GEMM another product.
// * The down product is launched with programmatic stream serialisation: its
//   blocks start as the up product's finish, request their first weight tiles,
//   and only then wait for H.
// Clusters are sized so that all blocks run at once, two per SM.  From 2 SMs of
// tiles on (f above 18944 on 148 SMs) a tile is one block and the rest of them
// run as the first ones leave: 8192 x 28672, one token (1409 MB, 448 up tiles)
// 223 us, 6.3 TB/s.
// Measured: one token, h = 4096, f = 14336 (352 MB of weights) 60 us, 5.8 TB/s
// over both products; 13 tokens, h = 2048, f = 5632 (69 MB) 23.6 us.  Tried on
// these: five stages 61 / 23.7 us, three 62 / 24.1; clusters up to 16 blocks
// 72 / 27; blocks of 4 warps, five per SM, 81 / 29; an even share of all slabs
// per block with partial sums through HBM, joined by the last block of a tile,
// 73 / 51.  Against the tcgen05 GEMM, whose 128-row tiles read the same
// weights: 32 tokens 82 against 84 us (h = 2048: 31 against 39), 64 tokens 150
// against 88 (52 against 40), so this path ends at 32 (too late for the widest
// blocks: 8192 x 28672, 32 tokens 288 us here, 33 by the GEMM 228).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "epi_math.cuh"
#include "stream_mma.cuh"
#include "tp_internal.h"

namespace tp {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kGroups = 4;  // K groups; kWarps / kGroups = 2 column runs
constexpr int kCols = 64;   // columns of a run
constexpr int kStepK = 16;
constexpr int kMaxCluster = 8;
constexpr int kMinSteps = 4;  // of a warp

struct ThinArgs {
  const __nv_bfloat16 *x, *w, *bias;
  __nv_bfloat16* out;       // up: the terms of H, [terms][M, N]
  __half* gu;   // [M, 2 N] or nullptr (up product)
  WaitCtl status;
  int M, K, N;              // N: columns of H, or of Z
  long long ldw;
  int act;
  int split;    // blocks per tile (the cluster)
  int pdl;      // wait for the previous kernel before reading x
};

template <int MT, int TERMS>
struct Cfg {
  static constexpr int kStages = 4;
  static constexpr int kWBytes = kStepK * kCols * 2;         // 2 KB
  static constexpr int kXTerm = MT * 16 * kStepK * 2;        // 512 bytes per 16 tokens
  static constexpr int kXBytes = TERMS * kXTerm;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kRed = kWarps * 16 * kCols * 4;       // one m-tile of every warp
  static constexpr int kSum = 2 * MT * 16 * kCols * 4;       // both runs, K groups added
  static constexpr int kBytes = kRing > kRed + kSum ? kRing : kRed + kSum;
};

__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

// Two values in fp16, saturated to its finite range.
__device__ __forceinline__ __half2 sat_half2(float2 v, bool& clamped) {
  if (fabsf(v.x) > kF16Max || fabsf(v.y) > kF16Max) {
    clamped = true;
    if (fabsf(v.x) > kF16Max) v.x = copysignf(kF16Max, v.x);
    if (fabsf(v.y) > kF16Max) v.y = copysignf(kF16Max, v.y);
  }
  return __floats2half2_rn(v.x, v.y);
}

template <int MT, bool GLU, int TERMS>
__global__ void __launch_bounds__(kThreads, 2) thin_product(const ThinArgs a) {
  using C = Cfg<MT, TERMS>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / a.split;
  const int run = warp & 1, kg = warp >> 1;
  const int col0 = tile * (GLU ? kCols : 2 * kCols) + (GLU ? 0 : run * kCols);  // output column
  const int ncols = min(kCols, a.N - col0);  // may be <= 0: the run is past the edge
  const __nv_bfloat16* w = a.w + col0 + (GLU ? run * static_cast<long long>(a.N) : 0);

  const int steps = (a.K + kStepK - 1) / kStepK;
  const int s0 = static_cast<int>(static_cast<long long>(steps) * rank / a.split) + kg;
  const int s1 = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / a.split);
  const int n = s0 < s1 ? (s1 - s0 + kGroups - 1) / kGroups : 0;

  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
  // Weight rows k .. k + 15 of this warp's i-th step: 16-byte chunk j of row r
  // at chunk j ^ (r & 7).
  auto fetch_w = [&](int i) {
    const uint32_t st = ring + (i % C::kStages) * C::kStageBytes;
    const int k = (s0 + i * kGroups) * kStepK;
    const int j = lane & 7;
    const bool okc = 8 * j + 8 <= ncols;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = x * 4 + (lane >> 3);
      const bool ok = okc && k + r < a.K;
      cp_async16(st + r * 128 + ((j ^ (r & 7)) << 4),
                 ok ? w + static_cast<long long>(k + r) * a.ldw + 8 * j : a.w, ok);
    }
  };
  // The tokens' values of the same K: 16-byte half h of token t (32-byte rows)
  // at half h ^ bit 2 of t.
  auto fetch_x = [&](int i) {
    const uint32_t st = ring + (i % C::kStages) * C::kStageBytes + C::kWBytes;
    const int k = (s0 + i * kGroups) * kStepK + 8 * (lane & 1);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int t = 16 * mt + (lane >> 1);
      const bool ok = t < a.M && k < a.K;
#pragma unroll
      for (int e = 0; e < TERMS; ++e)
        cp_async16(st + e * C::kXTerm + t * 32 + (((lane & 1) ^ ((t >> 2) & 1)) << 4),
                   ok ? a.x + (static_cast<long long>(e) * a.M + t) * a.K + k : a.x, ok);
    }
  };

#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i)
    if (i < n) fetch_w(i);
  pdl_next();
  if (a.pdl) pdl_wait();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (i < n) fetch_x(i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  float acc[MT][kCols / 8][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int c = 0; c < kCols / 8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][c][e] = 0.0f;

  const int wrow = (lane & 7) + (((lane >> 3) & 1) << 3), wcol = lane >> 4;
  const int xrow = lane & 15, xhalf = lane >> 4;
  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
    __syncwarp();  // all lanes' copies of this stage have landed; the stage
                   // fetched below has been read by every lane
    if (i + C::kStages - 1 < n) {
      fetch_w(i + C::kStages - 1);
      fetch_x(i + C::kStages - 1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const uint32_t sw = ring + (i % C::kStages) * C::kStageBytes, sx = sw + C::kWBytes;
    uint32_t xf[TERMS][MT][4];
#pragma unroll
    for (int e = 0; e < TERMS; ++e)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int t = 16 * mt + xrow;
        ldmatrix4<false>(xf[e][mt], sx + e * C::kXTerm + t * 32 + ((xhalf ^ ((t >> 2) & 1)) << 4));
      }
#pragma unroll
    for (int c = 0; c < kCols / 16; ++c) {
      uint32_t b[4];
      ldmatrix4<true>(b, sw + wrow * 128 + (((2 * c + wcol) ^ (wrow & 7)) << 4));
#pragma unroll
      for (int e = 0; e < TERMS; ++e)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816<true>(acc[mt][2 * c], xf[e][mt], b[0], b[1]);
          mma16816<true>(acc[mt][2 * c + 1], xf[e][mt], b[2], b[3]);
        }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // Add the K groups, 16 tokens at a time.
  float* red = reinterpret_cast<float*>(smem);                    // [warp][16][kCols]
  float* sum = reinterpret_cast<float*>(smem + C::kRed);          // [run][16 MT][kCols]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();  // the rings / the previous tokens' values are done with
#pragma unroll
    for (int c = 0; c < kCols / 8; ++c) {
      float* d = red + (warp * 16 + (lane >> 2)) * kCols + 8 * c + 2 * (lane & 3);
      *reinterpret_cast<float2*>(d) = make_float2(acc[mt][c][0], acc[mt][c][1]);
      *reinterpret_cast<float2*>(d + 8 * kCols) = make_float2(acc[mt][c][2], acc[mt][c][3]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * 16 * kCols / 2; x += kThreads) {
      const int rn = x / (16 * kCols / 2), y = x - rn * (16 * kCols / 2);
      float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        const float2 v = reinterpret_cast<const float2*>(red + (2 * q + rn) * 16 * kCols)[y];
        s.x += v.x;
        s.y += v.y;
      }
      reinterpret_cast<float2*>(sum + (rn * MT + mt) * 16 * kCols)[y] = s;
    }
  }
  if (a.split > 1)
    cluster_sync();
  else
    __syncthreads();

  // The tile's slices, in rank order; each block finishes its share of the
  // column pairs.
  const uint32_t base = smem_u32(sum);
  auto total = [&](int rn, int t, int c) {
    const uint32_t off = base + static_cast<uint32_t>(((rn * MT * 16 + t) * kCols + c) * 4);
    float2 s = make_float2(0.0f, 0.0f);
    for (int r = 0; r < a.split; ++r) {
      const float2 v = a.split > 1 ? ld_cluster2(mapa_shared(off, r))
                                   : *reinterpret_cast<const float2*>(
                                         sum + (rn * MT * 16 + t) * kCols + c);
      s.x += v.x;
      s.y += v.y;
    }
    return s;
  };
  auto bias2 = [&](int col) {
    if (a.bias == nullptr) return make_float2(0.0f, 0.0f);
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.bias + col));
  };
  const int pairs = (GLU ? kCols : 2 * kCols) / 2;
  const int tcol = tile * 2 * pairs;  // first output column of the tile
  for (int x = rank * kThreads + threadIdx.x; x < a.M * pairs; x += a.split * kThreads) {
    const int t = x / pairs, c = 2 * (x - t * pairs);
    const int col = tcol + c;
    if (col >= a.N) continue;
    if (GLU) {
      float2 g = total(0, t, c), u = total(1, t, c);
      const float2 bg = bias2(col), bu = bias2(a.N + col);
      g.x += bg.x;
      g.y += bg.y;
      u.x += bu.x;
      u.y += bu.y;
      if (a.gu != nullptr) {
        __half* p = a.gu + static_cast<long long>(t) * 2 * a.N + col;
        bool clamped = false;
        *reinterpret_cast<__half2*>(p) = sat_half2(g, clamped);
        *reinterpret_cast<__half2*>(p + a.N) = sat_half2(u, clamped);
        // A warp holds the 64 columns of one token, lanes past N left out; the
        // largest values of each 32, in 16 lanes.
        static_assert(kCols == 64, "a warp's columns");
        const int here = min(32, (a.N - tcol) / 2);
        const unsigned mask = 0xffffffffu >> (32 - here);
        float mg = fmaxf(fabsf(g.x), fabsf(g.y)), mu = fmaxf(fabsf(u.x), fabsf(u.y));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          const float vg = __shfl_xor_sync(mask, mg, o), vu = __shfl_xor_sync(mask, mu, o);
          if ((lane ^ o) < here) {
            mg = fmaxf(mg, vg);
            mu = fmaxf(mu, vu);
          }
        }
        const int bits = (clamped ? kFlagF16Range : 0) |
                         (f16_too_small(mg) || f16_too_small(mu) ? kFlagF16Small : 0);
        if (bits) status_flag(a.status, bits);
      }
      const float2 h = __fmul2_rn(gate_act2(g, a.act), u);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(h.x, h.y);
      __nv_bfloat16* p = a.out + static_cast<long long>(t) * a.N + col;
      *reinterpret_cast<__nv_bfloat162*>(p) = hi;
      if (a.M <= kThinTwoTermM) {
        const float2 hf = __bfloat1622float2(hi);
        *reinterpret_cast<__nv_bfloat162*>(p + static_cast<long long>(a.M) * a.N) =
            __floats2bfloat162_rn(h.x - hf.x, h.y - hf.y);
      }
    } else {
      float2 z = total(c / kCols, t, c % kCols);
      const float2 b = bias2(col);
      *reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<long long>(t) * a.N + col) =
          __floats2bfloat162_rn(z.x + b.x, z.y + b.y);
    }
  }
  if (a.split > 1) {
    __syncwarp();
    cluster_sync();  // no block leaves while its sums are read
  }
}

// Blocks per tile: the largest cluster with which all blocks still run at
// once (two per SM) and every warp keeps a few steps.
int plan_split(int tiles, int K) {
  const int64_t steps = (K + kStepK - 1) / kStepK;
  const int64_t fit = 2LL * sm_count() / tiles;
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({kMaxCluster, fit, steps / (kGroups * kMinSteps)})));
}

template <int MT, bool GLU, int TERMS>
tp_status launch(ThinArgs a, bool pdl, cudaStream_t stream) {
  constexpr int smem = Cfg<MT, TERMS>::kBytes;
  auto kern = thin_product<MT, GLU, TERMS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  // One carve-out for all of them: an SM that has to change it drains first, and
  // the down product's blocks would not start beside the up product's (72 us
  // for one token).
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return cuda_fail(e, "thin product smem");
  const int width = GLU ? kCols : 2 * kCols;
  const int tiles = (a.N + width - 1) / width;
  a.split = plan_split(tiles, a.K);
  a.pdl = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * a.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (a.split > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = a.split;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  const double cols = (GLU ? 2.0 : 1.0) * a.N;
  LaunchScope scope(TP_KIND_GEMM_STREAM, 2.0 * a.M * a.K * cols,
                    2.0 * (a.K * cols + double(a.M) * a.K + double(a.M) * a.N), stream, 1, 16 * MT,
                    a.M, a.N, a.K);
  e = cudaLaunchKernelEx(&cfg, kern, a);
  return e == cudaSuccess ? TP_OK : cuda_fail(e, "thin product launch");
}

template <bool GLU>
tp_status launch_m(const ThinArgs& a, bool pdl, cudaStream_t stream) {
  if (!GLU && a.M <= kThinTwoTermM) return launch<1, GLU, GLU ? 1 : 2>(a, pdl, stream);
  return a.M <= 16 ? launch<1, GLU, 1>(a, pdl, stream) : launch<2, GLU, 1>(a, pdl, stream);
}

}  // namespace

tp_status launch_thin_glu(const ThinGlu& g, cudaStream_t stream) {
  ThinArgs a{};
  a.M = static_cast<int>(g.M);
  a.act = g.act;
  a.x = static_cast<const __nv_bfloat16*>(g.x);
  a.w = static_cast<const __nv_bfloat16*>(g.wgu);
  a.bias = static_cast<const __nv_bfloat16*>(g.bgu);
  a.out = static_cast<__nv_bfloat16*>(g.H);
  a.gu = static_cast<__half*>(g.gu);
  if (a.gu != nullptr) {
    a.status = wait_ctl();
    if (a.status.st == nullptr) return fail(TP_ERR_CUDA, "device status unavailable");
  }
  a.K = static_cast<int>(g.h);
  a.N = static_cast<int>(g.f);
  a.ldw = 2 * g.f;
  tp_status s = launch_m<true>(a, false, stream);
  if (s != TP_OK) return s;
  a.x = static_cast<const __nv_bfloat16*>(g.H);
  a.w = static_cast<const __nv_bfloat16*>(g.wd);
  a.bias = static_cast<const __nv_bfloat16*>(g.bd);
  a.out = static_cast<__nv_bfloat16*>(g.z);
  a.gu = nullptr;
  a.K = static_cast<int>(g.f);
  a.N = static_cast<int>(g.h);
  a.ldw = g.h;
  return launch_m<false>(a, true, stream);
}

}  // namespace tp
