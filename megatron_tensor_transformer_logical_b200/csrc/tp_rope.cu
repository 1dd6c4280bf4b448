// Per-head RMS norm of queries and keys with the rotary position in the same
// pass, forward and backward.
//
// For a head's row x of d values, weight g and the token's position p:
//   r = 1 / sqrt(mean(x^2) + eps),  z = x r g            (norm; z = x without)
//   y_a = z_a cos t - z_b sin t,  y_b = z_b cos t + z_a sin t,  t = p f_i
// over the pairs (a, b) = (i, i + R/2) of the first R = d_rot values, or
// (2i, 2i + 1) when interleaved; the values past R pass through.  Backward,
// with dz the rotation of dy by -t:
//   dg = sum over rows of dz x r,
//   dx = r dz g - x r^3 mean(dz g x)
// r is recomputed from x, which the backward reads anyway, so the forward
// saves nothing.
//
// Both directions are HBM-bound: 2 elements moved per value forward, 3
// backward, about ten fp32 operations each.  The work is a list of units, a
// few neighbouring heads of one token (2 KB), and every warp takes a run of
// the list: it streams its units through its own ring of cp.async stages, so
// the bytes in flight do not depend on registers and nothing waits on a block
// barrier.  A row takes d / 8 lanes, 8 values per lane; a lane keeps its
// columns' cosines, with the weights folded in, in registers for all heads of
// a token, and reads the other value of each pair from shared memory.  The
// angles are formed once per token and warp, in fp64 (p f_i reduced by whole
// turns: an fp32 product would be off by radians at far positions).
// Measured at 8192 tokens of 32 + 8 heads of 128 in bf16 (168 MB forward, 252
// MB backward): 80 us for both, 5.2 TB/s; the issue of about 75 (backward 120)
// instructions per 16-byte piece and lane is what is left next to the HBM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "tp_internal.h"

namespace tp {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kMaxRot = 256;  // d <= 256
constexpr int kBlocksPerSm = 2;  // three would spill: 128 us instead of 80 (case below)

struct RopeSide {     // the query or the key heads
  const void* x;      // [M, heads * d], row stride ldx
  const void* dy;     // backward: gradient of the output
  void* out;          // y, or dx
  const void* g;      // [d] or nullptr
  long long ldx, lddy, ldo;
  int heads;
};

struct RopeArgs {
  RopeSide q, k;
  const int* pos;
  const double* inv_freq;
  float* part;        // backward: [blocks][2][d] partial weight gradients
  long long M;
  int d, d_rot, norm, interleaved;
  int uq, uk;         // units of one token: query heads, key heads
  long long units, per_warp;
  float eps;
};

// Eight values of a row in the storage type, as 32-bit words.
template <typename T>
struct Vec8 {
  static constexpr int kWords = sizeof(T) == 4 ? 8 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const;
  __device__ __forceinline__ void set(const float (&f)[8]);
};
template <>
__device__ __forceinline__ void Vec8<float>::get(float (&f)[8]) const {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
template <>
__device__ __forceinline__ void Vec8<float>::set(const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
}
template <>
__device__ __forceinline__ void Vec8<__nv_bfloat16>::get(float (&f)[8]) const {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <>
__device__ __forceinline__ void Vec8<__nv_bfloat16>::set(const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
}
template <>
__device__ __forceinline__ void Vec8<__half>::get(float (&f)[8]) const {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <>
__device__ __forceinline__ void Vec8<__half>::set(const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 t = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
}

// cos and sin of pos * f: the product in turns is reduced in fp64 to
// [-1/2, 1/2], then evaluated in fp32 with a first-order term for what the
// conversion to fp32 drops.
__device__ __forceinline__ float2 angle_cs(int pos, double f) {
  double u = static_cast<double>(pos) * f * 0.15915494309189533577;  // turns
  u = 2.0 * (u - rint(u));                                           // half turns
  const float uf = static_cast<float>(u);
  const float du = static_cast<float>(u - static_cast<double>(uf)) * 3.14159265358979f;
  float s, c;
  sincospif(uf, &s, &c);
  return make_float2(fmaf(-s, du, c), fmaf(c, du, s));
}

template <typename T, int LANES, bool BWD>
struct RopeCfg {
  static constexpr int kRows = 32 / LANES;                  // rows a warp holds at a time
  static constexpr int kSteps = sizeof(T) == 4 ? 2 : 4;     // such steps per unit
  static constexpr int kHeads = kRows * kSteps;             // heads per unit
  static constexpr int kPart = kHeads * LANES * 8 * sizeof(T);  // bytes of one operand, at most
  static constexpr int kUnit = (BWD ? 2 : 1) * kPart;       // x, and dy
  static constexpr int kStages = BWD ? 2 : 4;
  static constexpr int kRing = kStages * kUnit;             // per warp
  static constexpr int kCs = kMaxRot / 2 * 8;               // cos / sin of one token
  static constexpr int kSmem = kRopeWarps * (kRing + kCs);
};

__device__ __forceinline__ float2 swap2(float2 v) { return make_float2(v.y, v.x); }

template <typename T>
__device__ __forceinline__ void lds8(const uint8_t* p, float2 (&f)[4]) {
  Vec8<T> v;
  v.load(reinterpret_cast<const T*>(p));
  float t[8];
  v.get(t);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(t[2 * i], t[2 * i + 1]);
}

// IL: interleaved pairs; NORM: with the norm.
template <typename T, int LANES, bool BWD, bool IL, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, kBlocksPerSm) rope_kernel(const RopeArgs a) {
  using C = RopeCfg<T, LANES, BWD>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane & (LANES - 1), sub = lane / LANES, col = 8 * c;
  const int half = a.d_rot / 2;
  const bool on = col < a.d;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  uint8_t* ring = smem + warp * (C::kRing + C::kCs);
  float2* s_cs = reinterpret_cast<float2*>(ring + C::kRing);

  // The lane's part in the rotation: the columns of the pairs' other values
  // and the sign of their term.
  const bool rotated = col < a.d_rot;
  int pcol = on ? col : 0;
  float psign = 1.0f;
  if (rotated && !IL) {
    pcol = col < half ? col + half : col - half;
    psign = col < half ? -1.0f : 1.0f;
  }
  // byte offsets: the lane's columns in the first row of a step, its pairs'
  // other values from there, and the step to the next rows
  const int lane_off = (sub * a.d + (on ? col : 0)) * static_cast<int>(sizeof(T));
  const int partner_off = (pcol - (on ? col : 0)) * static_cast<int>(sizeof(T));
  const int step_bytes = C::kRows * a.d * static_cast<int>(sizeof(T));
  double freq[kMaxRot / 64];
#pragma unroll
  for (int i = 0; i < kMaxRot / 64; ++i)
    freq[i] = lane + 32 * i < half ? a.inv_freq[lane + 32 * i] : 0.0;

  const long long u0 = (static_cast<long long>(blockIdx.x) * kRopeWarps + warp) * a.per_warp;
  const long long u1 = min(u0 + a.per_warp, a.units);
  const int upt = a.uq + a.uk;

  // The walk over the units: token, unit within the token.
  struct Walk {
    long long m;
    int r;
  };
  auto at = [&](long long u) {
    Walk w;
    w.m = u / upt;
    w.r = static_cast<int>(u - w.m * upt);
    return w;
  };
  auto step = [&](Walk& w) {
    if (++w.r == upt) {
      w.r = 0;
      ++w.m;
    }
  };

  // A unit's rows are neighbours in memory: 16-byte pieces, dy behind x.
  auto fetch = [&](const Walk& w, int stage) {
    const bool key = w.r >= a.uq;
    const RopeSide& sd = key ? a.k : a.q;
    const int h0 = (key ? w.r - a.uq : w.r) * C::kHeads;
    const int bytes = min(C::kHeads, sd.heads - h0) * a.d * static_cast<int>(sizeof(T));
    const uint32_t dst = smem_u32(ring + stage * C::kUnit);
    const uint8_t* x = static_cast<const uint8_t*>(sd.x) +
                       (w.m * sd.ldx + static_cast<long long>(h0) * a.d) * sizeof(T);
    const uint8_t* dy = BWD ? static_cast<const uint8_t*>(sd.dy) +
                                  (w.m * sd.lddy + static_cast<long long>(h0) * a.d) * sizeof(T)
                            : nullptr;
#pragma unroll
    for (int i = 0; i < C::kPart / 512; ++i) {
      const int o = (i * 32 + lane) * 16;
      if (o < bytes) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + o), "l"(x + o)
                     : "memory");
        if (BWD)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + C::kPart + o),
                       "l"(dy + o)
                       : "memory");
      }
    }
  };

  Walk ahead = at(min(u0, a.units));
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (u0 + i < u1) {
      fetch(ahead, i);
      step(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // Columns 2 i and 2 i + 1 of the lane.  cs, sn: y = z cs + zp sn with zp the
  // pairs' other values (cs = 1, sn = 0 where nothing rotates; backward: the
  // opposite angle).  Forward: ca =
  // g cs, cb = gp sn, so y = r (x ca + xp cb); backward: ca = g.
  constexpr float rsign = BWD ? -1.0f : 1.0f;
  float2 cs[4], sn[4], ca[4], cb[4], dgq[4], dgk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = make_float2(1.0f, 1.0f);
    sn[i] = make_float2(0.0f, 0.0f);
    dgq[i] = dgk[i] = make_float2(0.0f, 0.0f);
  }
  auto side_weights = [&](const RopeSide& sd) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ca[i] = BWD ? make_float2(1.0f, 1.0f) : cs[i];
      cb[i] = sn[i];
    }
    if (!NORM || sd.g == nullptr || !on) return;
    float2 g[4], gp[4];
    lds8<T>(static_cast<const uint8_t*>(sd.g) + col * sizeof(T), g);
    if (!BWD && !IL) lds8<T>(static_cast<const uint8_t*>(sd.g) + pcol * sizeof(T), gp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BWD || IL) gp[i] = swap2(g[i]);
      ca[i] = __fmul2_rn(ca[i], g[i]);
      cb[i] = __fmul2_rn(cb[i], gp[i]);
    }
  };

  Walk w = at(min(u0, a.units));
  long long m_now = -1;
  bool key_now = false;
  int pos_next = u0 < u1 && half > 0 ? a.pos[w.m] : 0;
  int stage = 0;
  for (long long u = u0; u < u1; ++u) {
    const bool key = w.r >= a.uq;
    const RopeSide& sd = key ? a.k : a.q;
    if (w.m != m_now) {
      if (half > 0) {
        const int pos = pos_next;
        if (w.m + 1 < a.M) pos_next = a.pos[w.m + 1];
        __syncwarp();  // the last token's angles have been read
#pragma unroll
        for (int i = 0; i < kMaxRot / 64; ++i)
          if (lane + 32 * i < half) s_cs[lane + 32 * i] = angle_cs(pos, freq[i]);
        __syncwarp();
        if (rotated) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (IL) {
              const float2 v = s_cs[col / 2 + i];
              cs[i] = make_float2(v.x, v.x);
              sn[i] = make_float2(-rsign * v.y, rsign * v.y);
            } else {
              const int j = (col < half ? col : col - half) + 2 * i;
              const float2 v0 = s_cs[j], v1 = s_cs[j + 1];
              cs[i] = make_float2(v0.x, v1.x);
              sn[i] = make_float2(rsign * psign * v0.y, rsign * psign * v1.y);
            }
          }
        }
      }
      side_weights(sd);
    } else if (key != key_now) {
      side_weights(sd);
    }
    m_now = w.m;
    key_now = key;

    asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
    __syncwarp();  // all lanes' pieces of this stage have landed; the stage
                   // fetched below has been read by every lane
    if (u + C::kStages - 1 < u1) {
      fetch(ahead, stage == 0 ? C::kStages - 1 : stage - 1);
      step(ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");

    const int h0 = (key ? w.r - a.uq : w.r) * C::kHeads;
    // Rows past the heads and columns past d hold whatever an earlier unit
    // left: they enter no sum and are not stored.
    const uint8_t* px = ring + stage * C::kUnit + lane_off;
    uint8_t* po = static_cast<uint8_t*>(sd.out) +
                  (w.m * sd.ldo + static_cast<long long>(h0 + sub) * a.d + col) * sizeof(T);
#pragma unroll
    for (int s = 0; s < C::kSteps; ++s, px += step_bytes, po += step_bytes) {
      const int left = sd.heads - h0 - s * C::kRows;  // rows of this step
      if (left <= 0) break;
      const bool live = on && sub < left;
      float2 x[4], p[4], y[4];
      if constexpr (!BWD) {
        lds8<T>(px, x);
        if (!IL) lds8<T>(px + partner_off, p);
        float r = 1.0f;
        if (NORM) {
          float2 ss = __fmul2_rn(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) ss = __ffma2_rn(x[i], x[i], ss);
          float v = on ? ss.x + ss.y : 0.0f;
#pragma unroll
          for (int q = LANES / 2; q > 0; q >>= 1) v += __shfl_xor_sync(0xffffffffu, v, q);
          r = rsqrtf(fmaf(v, inv_d, a.eps));
        }
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (IL) p[i] = swap2(x[i]);
          y[i] = __ffma2_rn(x[i], ca[i], __fmul2_rn(p[i], cb[i]));
          if (NORM) y[i] = __fmul2_rn(r2, y[i]);
        }
      } else {
        float2 dz[4];
        lds8<T>(px + C::kPart, dz);
        if (!IL) lds8<T>(px + C::kPart + partner_off, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (IL) p[i] = swap2(dz[i]);
          dz[i] = __ffma2_rn(dz[i], cs[i], __fmul2_rn(p[i], sn[i]));
          y[i] = dz[i];
        }
        if (NORM) {
          lds8<T>(px, x);
          float2 ss = __fmul2_rn(x[0], x[0]), t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = __fmul2_rn(dz[i], x[i]);
          float2 dot = __fmul2_rn(t[0], ca[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            ss = __ffma2_rn(x[i], x[i], ss);
            dot = __ffma2_rn(t[i], ca[i], dot);
          }
          float s0 = on ? ss.x + ss.y : 0.0f, s1 = on ? dot.x + dot.y : 0.0f;
#pragma unroll
          for (int q = LANES / 2; q > 0; q >>= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, q);
            s1 += __shfl_xor_sync(0xffffffffu, s1, q);
          }
          const float r = rsqrtf(fmaf(s0, inv_d, a.eps));
          const float k = -s1 * inv_d * r * r * r;
          const float2 r2 = make_float2(r, r), k2 = make_float2(k, k);
          if (live) {
            if (key) {
#pragma unroll
              for (int i = 0; i < 4; ++i) dgk[i] = __ffma2_rn(t[i], r2, dgk[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) dgq[i] = __ffma2_rn(t[i], r2, dgq[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = __ffma2_rn(r2, __fmul2_rn(dz[i], ca[i]), __fmul2_rn(k2, x[i]));
        }
      }
      if (live) {
        const float f[8] = {y[0].x, y[0].y, y[1].x, y[1].y, y[2].x, y[2].y, y[3].x, y[3].y};
        Vec8<T> v;
        v.set(f);
        v.store(reinterpret_cast<T*>(po));
      }
    }
    if (++stage == C::kStages) stage = 0;
    step(w);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  if constexpr (BWD) {
    if (a.part == nullptr) return;
    // The block's weight gradients: the rows of a warp by shuffles, the warps
    // through shared memory in warp order, one partial row per block.
    __syncthreads();  // the rings are done with
    float* s_dg = reinterpret_cast<float*>(smem);  // [warp][query / key][kMaxRot]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) {
        dgq[i].x += __shfl_xor_sync(0xffffffffu, dgq[i].x, o);
        dgq[i].y += __shfl_xor_sync(0xffffffffu, dgq[i].y, o);
        dgk[i].x += __shfl_xor_sync(0xffffffffu, dgk[i].x, o);
        dgk[i].y += __shfl_xor_sync(0xffffffffu, dgk[i].y, o);
      }
      if (lane < LANES && on) {
        float* d = s_dg + warp * 2 * kMaxRot + col + 2 * i;
        *reinterpret_cast<float2*>(d) = dgq[i];
        *reinterpret_cast<float2*>(d + kMaxRot) = dgk[i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += kRopeThreads) {
      const int side = i / a.d, cc = i - side * a.d;
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kRopeWarps; ++q) s += s_dg[(q * 2 + side) * kMaxRot + cc];
      a.part[static_cast<long long>(blockIdx.x) * 2 * a.d + i] = s;
    }
  }
}

// dg[side][col] = sum over the blocks' partials, in a fixed order: 32 columns
// per block, 32 row phases each added in row order, the phases in phase order.
template <typename T>
__global__ void __launch_bounds__(1024) rope_dg_kernel(const float* part, int blocks, int d,
                                                       T* dgq, T* dgk) {
  __shared__ float s[32][33];
  const int cx = threadIdx.x & 31, ph = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + cx;
  float acc = 0.0f;
  if (i < 2 * d) {
#pragma unroll 8
    for (int b = ph; b < blocks; b += 32) acc += part[static_cast<long long>(b) * 2 * d + i];
  }
  s[ph][cx] = acc;
  __syncthreads();
  if (ph != 0 || i >= 2 * d) return;
  float t = 0.0f;
#pragma unroll
  for (int p = 0; p < 32; ++p) t += s[p][cx];
  T* dst = i < d ? dgq : dgk;
  if (dst != nullptr) dst[i < d ? i : i - d] = static_cast<T>(t);
}

// The persistent grid: the blocks that run at once.
int rope_max_blocks() { return kBlocksPerSm * sm_count(); }

template <typename T, int LANES, bool BWD>
tp_status launch(RopeArgs a, int* blocks, cudaStream_t stream) {
  using C = RopeCfg<T, LANES, BWD>;
  a.uq = (a.q.heads + C::kHeads - 1) / C::kHeads;
  a.uk = (a.k.heads + C::kHeads - 1) / C::kHeads;
  a.units = a.M * (a.uq + a.uk);
  const long long warps = static_cast<long long>(rope_max_blocks()) * kRopeWarps;
  a.per_warp = (a.units + warps - 1) / warps;
  *blocks = static_cast<int>((a.units + a.per_warp * kRopeWarps - 1) / (a.per_warp * kRopeWarps));
  auto kern = a.interleaved ? (a.norm ? rope_kernel<T, LANES, BWD, true, true>
                                      : rope_kernel<T, LANES, BWD, true, false>)
                            : (a.norm ? rope_kernel<T, LANES, BWD, false, true>
                                      : rope_kernel<T, LANES, BWD, false, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return cuda_fail(e, "query/key norm and rotary smem");
  kern<<<*blocks, kRopeThreads, C::kSmem, stream>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? TP_OK : cuda_fail(e, "query/key norm and rotary launch");
}

template <typename T, bool BWD>
tp_status launch_t(const RopeArgs& a, int* blocks, cudaStream_t stream) {
  if (a.d <= 64) return launch<T, 8, BWD>(a, blocks, stream);
  if (a.d <= 128) return launch<T, 16, BWD>(a, blocks, stream);
  return launch<T, 32, BWD>(a, blocks, stream);
}

template <typename T>
tp_status launch_b(const RopeArgs& a, bool bwd, int* blocks, cudaStream_t stream) {
  return bwd ? launch_t<T, true>(a, blocks, stream) : launch_t<T, false>(a, blocks, stream);
}

}  // namespace

size_t qk_rope_bwd_scratch_bytes(int64_t d) {
  return static_cast<size_t>(rope_max_blocks()) * 2 * static_cast<size_t>(d) * 4;
}

tp_status launch_qk_rope(const QkRope& r, bool bwd, void* scratch, cudaStream_t stream) {
  RopeArgs a{};
  a.q = {r.q, r.dqo, bwd ? r.dq : r.qo, r.gq, r.ldq, r.lddqo, bwd ? r.lddq : r.ldqo, r.heads};
  a.k = {r.k, r.dko, bwd ? r.dk : r.ko, r.gk, r.ldk, r.lddko, bwd ? r.lddk : r.ldko, r.kv_heads};
  a.pos = r.pos;
  a.inv_freq = r.inv_freq;
  a.M = r.M;
  a.d = r.d;
  a.d_rot = r.d_rot;
  a.norm = r.norm;
  a.interleaved = r.interleaved;
  a.eps = r.eps;
  const bool want_dg = bwd && r.norm && (r.dgq != nullptr || r.dgk != nullptr);
  a.part = want_dg ? static_cast<float*>(scratch) : nullptr;
  const double n = double(r.M) * (r.heads + r.kv_heads) * r.d;
  const double es = r.dtype == TP_F32 ? 4.0 : 2.0;
  int blocks = 0;
  if (r.M > 0) {
    LaunchScope scope(TP_KIND_REDUCE, (bwd ? 19.0 : 9.0) * n, (bwd ? 3.0 : 2.0) * n * es, stream);
    const tp_status st = r.dtype == TP_F32    ? launch_b<float>(a, bwd, &blocks, stream)
                         : r.dtype == TP_BF16 ? launch_b<__nv_bfloat16>(a, bwd, &blocks, stream)
                                              : launch_b<__half>(a, bwd, &blocks, stream);
    if (st != TP_OK) return st;
  }
  if (want_dg) {
    const int grid = (2 * r.d + 31) / 32;
    LaunchScope scope(TP_KIND_REDUCE, 2.0 * blocks * r.d, 8.0 * blocks * r.d, stream);
    const float* part = static_cast<const float*>(scratch);
    if (r.dtype == TP_F32)
      rope_dg_kernel<<<grid, 1024, 0, stream>>>(part, blocks, r.d, static_cast<float*>(r.dgq),
                                                static_cast<float*>(r.dgk));
    else if (r.dtype == TP_BF16)
      rope_dg_kernel<<<grid, 1024, 0, stream>>>(part, blocks, r.d,
                                                static_cast<__nv_bfloat16*>(r.dgq),
                                                static_cast<__nv_bfloat16*>(r.dgk));
    else
      rope_dg_kernel<<<grid, 1024, 0, stream>>>(part, blocks, r.d, static_cast<__half*>(r.dgq),
                                                static_cast<__half*>(r.dgk));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "norm weight gradient launch");
  }
  return TP_OK;
}

}  // namespace tp
