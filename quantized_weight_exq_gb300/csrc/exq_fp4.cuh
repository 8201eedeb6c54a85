// What the kernels of the microscaled 4-bit format share: its layout, the
// conversions between codes, scale bytes and numbers, and the wrappers of
// barriers and bulk copies.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "exq_internal.h"

namespace exq {

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == EXQ_FP4_E4M3 ? 16 : 32; }
// k values of one 512-byte scale tile (4 blocks)
__host__ __device__ constexpr int fp4_tile_k(int fmt) { return 4 * fp4_block(fmt); }

// byte of row r (0..127) in a scale tile; block j of the four is byte + j
__host__ __device__ constexpr int fp4_tile_byte(int r) { return (r & 31) * 16 + (r >> 5) * 4; }

// A launch that may begin while the one before it on the stream ends (a
// programmatic dependent): its kernel calls griddepcontrol.wait before it reads
// or writes memory.
template <typename... P, typename... A>
exq_status launch_dependent(void (*fn)(P...), int blocks, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...) == cudaSuccess ? EXQ_OK : EXQ_ERR_CUDA;
}

// ---------------------------------------------------------------- numbers

// the two e2m1 codes of byte B of w, as fp16 (exact; the even k in the low half)
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(r)
      : "r"(w), "n"(B));
  return r;
}

// 8 numbers -> 8 codes, to nearest even, at most 6; v[0] in the low nibble
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// the e2m1 number nearest to q (|q| <= 6) and its code
__device__ __forceinline__ void e2m1_nearest(float q, uint32_t& code, float& value) {
  uint32_t both;
  asm("{\n\t.reg .b8 b, z;\n\t.reg .b32 f;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, 0f00000000, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(code), "=r"(both)
      : "f"(q));
  value = __half2float(__ushort_as_half(static_cast<unsigned short>(both)));
}

// two e4m3 bytes (the low 16 bits) as fp16, exact; 0x7f is NaN
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t bytes) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(bytes));
  return r;
}

__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_f16(byte & 0xFFu))));
}

// two numbers -> e4m3 bytes, to nearest even, at most 448; hi in bits 8..15
__device__ __forceinline__ uint32_t e4m3x2(float hi, float lo) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// 2^(byte - 127), subnormal for 0, NaN for 255
__device__ __forceinline__ float e8m0_f32(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// ---------------------------------------------------------------- barriers and copies

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One lane of a converged warp. The code around it stays the whole warp's: the
// operands of tcgen05 instructions are uniform registers, and a loop that one
// lane runs alone brings each of them there anew (150 clocks an MMA, where the
// tensor core takes 46).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

constexpr int kFp4WaitLimit = 1 << 22;  // try_wait rounds before giving up

// Bounded wait of a whole warp (every lane tests; a vote keeps the lanes
// together). False, with the timeout recorded in *err and *abort_flag set for the
// CTA's other roles, if the phase does not complete.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int limit,
                                               unsigned* err) {
  for (int i = 0; i < limit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
  }
  if ((threadIdx.x & 31) == 0) {
    atomicOr(err, kDevErrTimeout);
    *abort_flag = 1;
  }
  __syncwarp();
  return false;
}

// Waits for the copies of the last n of the stages 0 .. issued - 1 that this warp has issued: all have landed before the CTA may
// exit. Each warp that issues copies waits for its own: after a timeout one may be ahead of another, and a stage that lacks the
// other's share does not complete. What is waited then is still a thousand times what a copy takes.
__device__ __forceinline__ void await_issued(const uint64_t* full, int issued, int n, int limit) {
  for (int i = max(0, issued - n); i < issued; ++i)
    for (int r = 0; r < min(limit, 1 << 16); ++r)
      if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(&full[i % n]), (i / n) & 1))) break;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// contiguous bytes (a multiple of 16, both addresses on 16-byte boundaries)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace exq
