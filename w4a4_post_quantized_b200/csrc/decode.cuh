// decode.cuh -- shared by the single-token operators (group.cu, kv.cu): the
// two 16-bit types and checks of arguments.
//
// The operators' kernels start while the one in front still writes, so they read with ordinary
// loads only, behind their wait: non-coherent ones (__ldg, const pointers marked __restrict__)
// are for memory that nothing writes during a kernel's lifetime.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "w4a4.h"

namespace w4a4 {
namespace {

// (a & b) ^ c in one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

struct Bf16 {
  // log2 of the largest softmax weight: the type's range is that of fp32
  static constexpr float kTop = 0.0f;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  // element 0 of a packed pair in the low half
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint16_t round(float a) { return __bfloat16_as_ushort(__float2bfloat16_rn(a)); }
  // The 8 codes of a word (4-bit two's complement, element 2 p in nibble p, 2 p + 1 in nibble p + 4) as 4 pairs:
  // 2^7 + u with u = c + 8 in the low mantissa bits, minus 136; exact.
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t v = and_xor(w >> (4 * p), 0x000F000Fu, 0x43084308u);
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[p]) : "r"(v), "r"(0x43084308u));
    }
  }
  // d (16 x 8) += A (16 x 16) B (16 x 8), fp32 sums
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // d = A B
  static __device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  }
};

struct Fp16 {
  // Weights go up to 2^15, so that those down to 2^-39 of the largest are held, to 2^-40 of it (2^-24 is the
  // least there is; 2^-26 of 1 would be lost, and a hundred thousand of those are 2^-9 of the sum).
  static constexpr float kTop = 15.0f;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ float lo(uint32_t w) { return to_f32(static_cast<uint16_t>(w & 0xFFFFu)); }
  static __device__ __forceinline__ float hi(uint32_t w) { return to_f32(static_cast<uint16_t>(w >> 16)); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint16_t round(float a) { return __half_as_ushort(__float2half_rn(a)); }
  // As above with 2^10 + u; the nibbles at bits 4..7 stand for 16 u.
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
    for (int p = 0; p < 4; p += 2) {
      const uint32_t v = w >> (4 * p);
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[p]) : "r"(and_xor(v, 0x000F000Fu, 0x64086408u)), "r"(0x64086408u));
      // (2^10 + 16 u) / 16 - 72
      asm("fma.rn.f16x2 %0, %1, %2, %3;"
          : "=r"(o[p + 1]) : "r"(and_xor(v, 0x00F000F0u, 0x64806480u)), "r"(0x2C002C00u), "r"(0xD480D480u));
    }
  }
  // d (16 x 8) += A (16 x 16) B (16 x 8), fp32 sums
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // d = A B
  static __device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  }
};

inline bool ptr_aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ptr_aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Whether any of `rows` runs of `row` elements, `stride` apart from a on, shares memory with the n elements at b.
inline bool overlap(const uint16_t *a, int64_t rows, int64_t row, int64_t stride, const uint16_t *b, int64_t n) {
  const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / 2;
  // the first run that ends behind b
  const int64_t t = at < row || stride == 0 ? 0 : (at - row) / stride + 1;
  return t < rows && t * stride + row > at && t * stride < at + n;
}
// Whether n bytes at a and m bytes at b share any.
inline bool overlap_bytes(const void *a, size_t n, const void *b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < n : x - y < m;
}
inline w4a4_status launch_status(cudaError_t e) { return e == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA; }

}  // namespace
}  // namespace w4a4
