// ptx_e4m3.cuh -- what products over e4m3 operands need beyond ptx.cuh: the
// MMA of 8-bit types, descriptors of 64-byte-swizzled operands, and numbers as
// two e4m3 parts.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace mha {

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, e4m3 inputs, K = 32.
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// Instruction descriptor, kind::f8f6f4 with e4m3 A/B (format 0) and fp32
// accumulator; the fields are those of idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn_major,
                                                      bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// The same of kind::f16 with fp16 A/B (format 0, too).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major,
                                                     bool b_mn_major) {
  return idesc_e4m3_f32(M, N, a_mn_major, b_mn_major);
}

// Shared-memory descriptor of an operand whose rows are kRowBytes (128 or 64)
// long and swizzled over as many: the fields are those of sdesc_sw128, with
// layout 4 for the 64-byte swizzle (atoms of 8 rows x 64 bytes, 512-byte
// aligned).
template <int kRowBytes>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo_bytes,
                                               uint32_t sbo_bytes) {
  static_assert(kRowBytes == 128 || kRowBytes == 64, "swizzle");
  const uint64_t d = sdesc_sw128(saddr, lbo_bytes, sbo_bytes);
  return kRowBytes == 128 ? d : (d & ~(7ull << 61)) | (4ull << 61);
}

// Byte offset of 16-byte piece c of row r in such an operand.
template <int kRowBytes>
__device__ __forceinline__ int piece_at(int r, int c) {
  if constexpr (kRowBytes == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// 32 lanes x 32 bit, 8 consecutive columns: to registers, with the wait in the
// same asm statement, and from them.
__device__ __forceinline__ void tmem_ld8_sync(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 32 lanes x 32 bit, 16 consecutive columns from 16 registers per thread.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// (lo, hi) to e4m3, to nearest, at most 448.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t u) {
  return __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u), __NV_E4M3)));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two numbers as two parts each, x = first + second / up: the first off by at
// most 2^-4 of x, the rest of it by 2^-4 of that, so together by 2^-8 (or by
// 2^-10 / up near zero); exact for 8-bit mantissas whose lowest bit is at
// least 2^-9 / up.  |x| up * 2^-4 <= 448.
__device__ __forceinline__ void two_parts(float a, float b, float up, uint32_t* first,
                                          uint32_t* second) {
  *first = to_e4m3x2(a, b);
  const float2 f = from_e4m3x2(*first);
  *second = to_e4m3x2((a - f.x) * up, (b - f.y) * up);
}

// The power of two s >= 2^-126 that brings a row's largest element x to at
// most 448 (and above 224 where it can), and its inverse.
__device__ __forceinline__ float part_scale_of(float x, float* inverse) {
  const unsigned u = __float_as_uint(x);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = x > 0.f ? max(e, -126) : 0;
  *inverse = __uint_as_float(static_cast<unsigned>(127 - e) << 23);
  return __uint_as_float(static_cast<unsigned>(e + 127) << 23);
}

}  // namespace mha
