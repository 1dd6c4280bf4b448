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
// backward, about ten fp32 operations each.  A row takes d / 8 lanes of a
// warp, 8 values (16 or 32 bytes) per lane; a lane keeps its columns' weights
// and cosines in registers while it walks the heads of one token, so a row
// costs its loads, two shuffle trees at most and one exchange of the raw
// values with the lane that holds the other half of its pairs.  The angles of
// a token are formed once per block, in fp64 (p f_i reduced by whole turns:
// an fp32 product would be off by radians at far positions), and shared by
// all heads.
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
constexpr int kRowsInFlight = 4;

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
  int wpt_log2;       // warps that share one token (log2)
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
  __device__ __forceinline__ void shuffle_from(const Vec8& o, int lane) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __shfl_sync(0xffffffffu, o.w[i], lane);
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

// Sum over the LANES lanes that hold one row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

// What a lane holds for its eight columns of the rotation.
struct LaneRot {
  float cs[8], sn[8];  // per column; sn carries the sign of the partner's term
  int partner;         // lane with the other half of the pairs (half-split form)
  bool rot;            // this lane's columns are rotated
};

// y = z rotated by sign * angle; zp: the partner lane's values (half-split).
__device__ __forceinline__ void rotate8(const float (&z)[8], const float (&zp)[8],
                                        const LaneRot& r, bool interleaved, float sign,
                                        float (&y)[8]) {
  if (!r.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = z[i];
  } else if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(z[i], r.cs[i], sign * r.sn[i] * z[i ^ 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(z[i], r.cs[i], sign * r.sn[i] * zp[i]);
  }
}

// One side's heads of one token.  hw: this warp's index among the warps of
// the token; LANES lanes per row, 32 / LANES rows per warp.
template <typename T, int LANES, bool BWD>
__device__ __forceinline__ void rope_heads(const RopeSide& sd, const RopeArgs& a, long long m,
                                           int hw, const LaneRot& rot, float (&dg)[8]) {
  constexpr int kRows = 32 / LANES;
  const int lane = threadIdx.x & 31;
  const int c = lane & (LANES - 1);
  const int sub = lane / LANES;
  const bool on = 8 * c < a.d;
  const int wpt = 1 << a.wpt_log2;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const bool il = a.interleaved != 0, norm = a.norm != 0;

  // weights of this lane's columns and (half-split forward) its partner's
  float g[8], gp[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = gp[i] = 1.0f;
  if (norm && sd.g != nullptr) {
    Vec8<T> gv, gpv;
    gv.zero();
    if (on) gv.load(static_cast<const T*>(sd.g) + 8 * c);
    gpv.shuffle_from(gv, rot.partner);
    gv.get(g);
    gpv.get(gp);
  }
  const T* xrow = static_cast<const T*>(sd.x) + m * sd.ldx + 8 * c;
  const T* dyrow = BWD ? static_cast<const T*>(sd.dy) + m * sd.lddy + 8 * c : nullptr;
  T* orow = static_cast<T*>(sd.out) + m * sd.ldo + 8 * c;

  constexpr int U = BWD ? kRowsInFlight / 2 : kRowsInFlight;
  for (int h0 = hw * kRows; h0 < sd.heads; h0 += U * wpt * kRows) {
    Vec8<T> x[U], dy[BWD ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * wpt * kRows + sub;
      x[u].zero();
      if (BWD) dy[u].zero();
      if (on && h < sd.heads) {
        x[u].load(xrow + static_cast<long long>(h) * a.d);
        if (BWD) dy[u].load(dyrow + static_cast<long long>(h) * a.d);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hb = h0 + u * wpt * kRows;  // warp-uniform
      if (hb >= sd.heads) break;
      const int h = hb + sub;
      float xf[8], y[8];
      x[u].get(xf);
      float r = 1.0f;
      if (norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(xf[i], xf[i], ss);
        r = rsqrtf(fmaf(row_sum<LANES>(ss), inv_d, a.eps));
      }
      Vec8<T> pv;
      float pf[8];
      if (!BWD) {
        pv.shuffle_from(x[u], rot.partner);
        pv.get(pf);
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z[i] = xf[i] * r * g[i];
          pf[i] = pf[i] * r * gp[i];
        }
        rotate8(z, pf, rot, il, 1.0f, y);
      } else {
        float dyf[8], dz[8];
        dy[u].get(dyf);
        pv.shuffle_from(dy[u], rot.partner);
        pv.get(pf);
        rotate8(dyf, pf, rot, il, -1.0f, dz);
        if (norm) {
          float dot = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (h < sd.heads) dg[i] = fmaf(dz[i], xf[i] * r, dg[i]);
            dz[i] *= g[i];
            dot = fmaf(dz[i], xf[i], dot);
          }
          const float k = row_sum<LANES>(dot) * inv_d * r * r * r;
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = fmaf(r, dz[i], -k * xf[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = dz[i];
        }
      }
      if (on && h < sd.heads) {
        Vec8<T> o;
        o.set(y);
        o.store(orow + static_cast<long long>(h) * a.d);
      }
    }
  }
}

// A block takes 8 >> wpt_log2 tokens at a time and strides over the groups.
template <typename T, int LANES, bool BWD>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 s_cs[kRopeWarps * (kMaxRot / 2)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpb = kRopeWarps >> a.wpt_log2;  // tokens per block
  const int half = a.d_rot / 2;
  const int tok = warp >> a.wpt_log2, hw = warp & ((1 << a.wpt_log2) - 1);
  const int c = lane & (LANES - 1);
  const bool il = a.interleaved != 0;

  LaneRot rot;
  rot.rot = 8 * c < a.d_rot;
  rot.partner = lane;
  float psign = 1.0f;  // the sign of the partner's term in the forward
  if (rot.rot && !il) {
    const bool first = 8 * c < half;
    rot.partner = first ? lane + half / 8 : lane - half / 8;
    psign = first ? -1.0f : 1.0f;
  }
  float dgq[8], dgk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dgq[i] = dgk[i] = 0.0f;

  const long long groups = (a.M + tpb - 1) / tpb;
  for (long long grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    for (int i = threadIdx.x; i < tpb * half; i += kRopeThreads) {
      const int t = i / half;
      const long long m = grp * tpb + t;
      if (m < a.M) s_cs[i] = angle_cs(a.pos[m], a.inv_freq[i - t * half]);
    }
    __syncthreads();
    const long long m = grp * tpb + tok;
    if (m < a.M) {
      if (rot.rot) {
        const float2* cs = s_cs + tok * half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          int j = 8 * c + i;
          float sg = psign;
          if (il) {
            sg = (j & 1) ? 1.0f : -1.0f;
            j >>= 1;
          } else if (j >= half) {
            j -= half;
          }
          rot.cs[i] = cs[j].x;
          rot.sn[i] = sg * cs[j].y;
        }
      }
      rope_heads<T, LANES, BWD>(a.q, a, m, hw, rot, dgq);
      if (a.k.heads > 0) rope_heads<T, LANES, BWD>(a.k, a, m, hw, rot, dgk);
    }
    __syncthreads();
  }

  if constexpr (BWD) {
    if (a.part == nullptr) return;
    // The block's weight gradients: the rows of a warp by shuffles, the warps
    // through shared memory in warp order, one partial row per block.
    __shared__ float s_dg[kRopeWarps][2][kMaxRot];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) {
        dgq[i] += __shfl_xor_sync(0xffffffffu, dgq[i], o);
        dgk[i] += __shfl_xor_sync(0xffffffffu, dgk[i], o);
      }
      if (lane < LANES && 8 * c < a.d) {
        s_dg[warp][0][8 * c + i] = dgq[i];
        s_dg[warp][1][8 * c + i] = dgk[i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += kRopeThreads) {
      const int side = i / a.d, col = i - side * a.d;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kRopeWarps; ++w) s += s_dg[w][side][col];
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
  if (i < 2 * d)
    for (int b = ph; b < blocks; b += 32) acc += part[static_cast<long long>(b) * 2 * d + i];
  s[ph][cx] = acc;
  __syncthreads();
  if (ph != 0 || i >= 2 * d) return;
  float t = 0.0f;
#pragma unroll
  for (int p = 0; p < 32; ++p) t += s[p][cx];
  T* dst = i < d ? dgq : dgk;
  if (dst != nullptr) dst[i < d ? i : i - d] = static_cast<T>(t);
}

// At most this many blocks run the backward, so the partials stay small: four
// per SM.
int rope_max_blocks() { return 4 * sm_count(); }

template <typename T, int LANES>
void launch(const RopeArgs& a, bool bwd, int blocks, cudaStream_t stream) {
  if (bwd)
    rope_kernel<T, LANES, true><<<blocks, kRopeThreads, 0, stream>>>(a);
  else
    rope_kernel<T, LANES, false><<<blocks, kRopeThreads, 0, stream>>>(a);
}

template <typename T>
void launch_t(const RopeArgs& a, bool bwd, int blocks, cudaStream_t stream) {
  if (a.d <= 64)
    launch<T, 8>(a, bwd, blocks, stream);
  else if (a.d <= 128)
    launch<T, 16>(a, bwd, blocks, stream);
  else
    launch<T, 32>(a, bwd, blocks, stream);
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
  // Few tokens: several warps share a token's heads, up to a block per token,
  // as long as that leaves no more than about two blocks per SM.
  const long long sms = sm_count();
  while (a.wpt_log2 < 3 && (r.M << (a.wpt_log2 + 1)) <= 2 * sms * kRopeWarps) ++a.wpt_log2;
  const long long tpb = kRopeWarps >> a.wpt_log2;
  const long long groups = (r.M + tpb - 1) / tpb;
  const int blocks = static_cast<int>(
      std::min<long long>(groups, bwd ? rope_max_blocks() : (1ll << 30)));
  const double n = double(r.M) * (r.heads + r.kv_heads) * r.d;
  const double es = r.dtype == TP_F32 ? 4.0 : 2.0;
  if (blocks > 0) {
    LaunchScope scope(TP_KIND_REDUCE, (bwd ? 19.0 : 9.0) * n, (bwd ? 3.0 : 2.0) * n * es, stream);
    if (r.dtype == TP_F32)
      launch_t<float>(a, bwd, blocks, stream);
    else if (r.dtype == TP_BF16)
      launch_t<__nv_bfloat16>(a, bwd, blocks, stream);
    else
      launch_t<__half>(a, bwd, blocks, stream);
  }
  cudaError_t e = cudaSuccess;
  if (blocks > 0 && (e = cudaGetLastError()) != cudaSuccess)
    return cuda_fail(e, "query/key norm and rotary launch");
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
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "norm weight gradient launch");
  }
  return TP_OK;
}

}  // namespace tp
