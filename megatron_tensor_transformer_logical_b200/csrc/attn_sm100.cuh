// Device helpers shared by the attention kernels on the sm_100a tensor cores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx_sm100.cuh"

namespace tp {

// kind::f16 instruction descriptor with fp16 A/B and fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(n) >> 3) << 17) | ((static_cast<uint32_t>(m) >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&t);
}

// Three-input maximum (one instruction on sm_100).
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// max(m, v[0..31]) by three-input maxima: 16 instructions, depth 4.
__device__ __forceinline__ float max32(const float (&v)[32], float m) {
  float w[12];
#pragma unroll
  for (int k = 0; k < 10; ++k) w[k] = max3f(v[3 * k], v[3 * k + 1], v[3 * k + 2]);
  w[10] = v[30];
  w[11] = v[31];
  float x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = max3f(w[3 * k], w[3 * k + 1], w[3 * k + 2]);
  return max3f(max3f(x[0], x[1], x[2]), x[3], m);
}

// Two warp-collective loads of 32 lanes x 32 columns with a single wait.
__device__ __forceinline__ void tmem_ld32x2(uint32_t ta, float (&va)[32], uint32_t tb,
                                            float (&vb)[32]) {
  uint32_t a[32], b[32];
#define TP_LD32(dst, addr)                                                                  \
  asm volatile(                                                                            \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "                                            \
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "            \
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "  \
      "[%32];"                                                                             \
      : "=r"(dst[0]), "=r"(dst[1]), "=r"(dst[2]), "=r"(dst[3]), "=r"(dst[4]),             \
        "=r"(dst[5]), "=r"(dst[6]), "=r"(dst[7]), "=r"(dst[8]), "=r"(dst[9]),             \
        "=r"(dst[10]), "=r"(dst[11]), "=r"(dst[12]), "=r"(dst[13]), "=r"(dst[14]),        \
        "=r"(dst[15]), "=r"(dst[16]), "=r"(dst[17]), "=r"(dst[18]), "=r"(dst[19]),        \
        "=r"(dst[20]), "=r"(dst[21]), "=r"(dst[22]), "=r"(dst[23]), "=r"(dst[24]),        \
        "=r"(dst[25]), "=r"(dst[26]), "=r"(dst[27]), "=r"(dst[28]), "=r"(dst[29]),        \
        "=r"(dst[30]), "=r"(dst[31])                                                       \
      : "r"(addr)                                                                          \
      : "memory")
  TP_LD32(a, ta);
  TP_LD32(b, tb);
#undef TP_LD32
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // The wait orders the loads; the copies below cannot move above it (the
  // asm is volatile with a memory clobber).
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    va[i] = __uint_as_float(a[i]);
    vb[i] = __uint_as_float(b[i]);
  }
}

// Issue by a whole converged warp, whose elected lane (the same each time)
// gives the instructions: descriptors and addresses then stay in uniform
// registers, where code under a branch to one lane moves them there for every
// product (about 85 clocks a product, more than one of 128 x 64 x 16 takes).
// Four products, K = 64: D (+)= A B, A and B in K-major tiles (16 columns 32
// bytes apart), `accumulate` for the first.
__device__ __forceinline__ void warp_umma_ss4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "setp.eq.b32 p, %4, %4;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in tensor memory, 16 columns of A in 8, the second 32 of them
// HALF columns on, and B an MN-major tile (16 rows of 128 bytes).
template <int HALF = 16>
__device__ __forceinline__ void warp_umma_ts4(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "setp.eq.b32 p, %4, %4;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, %1, %5;\n\tadd.s64 b, %2, 256;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, %1, %6;\n\tadd.s64 b, %2, 384;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "n"(HALF), "n"(HALF + 8)
      : "memory");
}

__device__ __forceinline__ void warp_umma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

// mbar_wait by a converged warp, which stays so.
__device__ __forceinline__ bool warp_mbar_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w,
                                               int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w, code));
}

// The block's last barrier.  Where a wait has given up, copies and products may
// still be under way: they get 200 us (they take a few) before tensor memory
// is freed and the block leaves its shared memory.
__device__ __forceinline__ void leave(bool gave_up) {
  if (__syncthreads_or(gave_up)) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) __nanosleep(1000);
    __syncthreads();
  }
}

// 3-D tiled load of one box (columns x, rows y of sequence z) into shared
// memory; completion is signalled on `bar` through its transaction count.
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x,
                                             int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

}  // namespace tp
