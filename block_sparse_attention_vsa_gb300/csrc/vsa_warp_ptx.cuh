// vsa_warp_ptx.cuh -- thin inline-PTX wrappers for the warp-level pieces of the block
// choice and 8-bit cache kernels: 16-byte asynchronous copies, the m16n8k16 tensor
// product, 8x8 transposes and e4m3 conversions.  Written from the public PTX ISA
// description of these instructions.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace vsa {

// A kernel launched with programmatic serialization starts while its predecessor in the
// stream still runs.  First thing in the kernel: wait until the predecessor has ended and
// its writes are visible, and let the successor start likewise.  Nothing is read or
// written before that, so the order of the stream's work is that of ordinary launches; what
// overlaps is the start-up, in which lines that the kernel will read may be fetched into L2
// (where all SMs' writes meet: a line fetched early is never stale).
__device__ __forceinline__ void after_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// What a call reads may be what its predecessor in the stream writes, and this kernel's life
// begins before that one's ends: not memory that is read-only for as long as the kernel
// lives, which the non-coherent path (__ldg, const __restrict__ parameters) asks for and
// which lets the compiler move a load above the wait.  These kernels read by ordinary loads,
// which stay behind the wait's memory clobber.
template <typename T>
__device__ __forceinline__ T read_global(const T* p) {
  return *p;
}

// `bytes` from `p` on into L2, a line a thread.
__device__ __forceinline__ void prefetch_l2(const void* p, size_t bytes, int tid, int threads) {
  for (size_t at = (size_t)tid * 128; at < bytes; at += (size_t)threads * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + at));
}

// 16 bytes global -> shared, asynchronously; `n_src` of them are read (0 or 16), the
// rest of the destination is filled with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst_smem, const void* src, uint32_t n_src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem),
               "l"(static_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(n_src)
               : "memory");
}
// 4 bytes global -> shared, asynchronously.
__device__ __forceinline__ void cp_async4(uint32_t dst_smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst_smem),
               "l"(static_cast<uint64_t>(__cvta_generic_to_global(src)))
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (+)= A * B, one m16n8k16 tile, fp32 accumulators.  With g = lane / 4, i = lane % 4:
//   A: a0 = (row g, k 2i..2i+1), a1 = (row g+8, same k), a2, a3 the same at k+8
//   B: b0 = (k 2i..2i+1, column g), b1 the same at k+8
//   D: d0, d1 = (row g, columns 2i, 2i+1), d2, d3 = (row g+8)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7},"
      " {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held one row of pairs per 4 lanes.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// The two halves of a word of four e4m3 values, each as two fp16 (exact).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// Two fp32 -> two e4m3 (nearest even; beyond +-448 saturates, NaN stays NaN); `lo` in
// bits 0..7.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two fp32 -> packed fp16x2 (nearest even); `lo` in bits 0..15.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// acc_lo += fp16 value in bits 0..15 of w, acc_hi += fp16 value in bits 16..31 (fp32 adds of
// the exact values, no unpacking)
__device__ __forceinline__ void add_f16x2_to_f32(uint32_t w, float& acc_lo, float& acc_hi) {
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n add.rn.f32.f16 %0, lo, %0;\n"
      " add.rn.f32.f16 %1, hi, %1;\n}"
      : "+f"(acc_lo), "+f"(acc_hi)
      : "r"(w));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

}  // namespace vsa
