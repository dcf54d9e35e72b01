// Device helpers for microscaled 4-bit floats (MX4), shared by the kernels that read them.
//
// A value is e2m1(code) * 2^(s - 127): code bits are sign, two of exponent, one of mantissa
// (0, 0.5, 1, 1.5, 2, 3, 4, 6), and one byte s is shared by 32 consecutive inputs of a row.  A
// block of 32 codes is 16 bytes, so one 128-bit load holds exactly one block of one row and one
// scale; a "chunk" is 128 inputs (four blocks, and the aligned dword of their four scales).
//
// Both matrix instructions used here take their operands as lane (q, r) = (lane / 16, lane % 16)
// holding row r, block q of a chunk:
//  - v_mfma_scale_f32_16x16x128_f8f6f4 reads the block's codes and scale byte as they are stored;
//  - v_mfma_f32_16x16x32_bf16 takes eight inputs per lane; instruction j of a chunk takes codes
//    8j .. 8j+7 of every lane's block, so its 32 inputs are 128c + 32q + 8j .. +7 over q (the
//    order of a sum's terms is free as long as both operands use it).
// The bf16 operands are exact: a code times a power of two keeps two significant bits, bf16 has
// fp32's exponent range, and its subnormals (s = 0) are multiplied, not flushed.  s = 255 is NaN.
#pragma once

#include "ql_internal.hpp"
#include "ql_stream.hpp"

namespace ql {

constexpr int kMxBlock = 32;   // inputs per scale
constexpr int kMxChunk = 128;  // inputs per chunk: four blocks

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

typedef const __attribute__((address_space(1))) uint32_t* mx_gu32p;

__host__ __device__ inline int64_t mx4_scale_stride(int64_t K) { return (K + kMxChunk - 1) / kMxChunk * 4; }

// 16 bytes at p (global memory)
__device__ __forceinline__ u32x4_t ld_b128(const void* p) { return *(gu32x4p)p; }
__device__ __forceinline__ uint32_t ld_b32(const void* p) { return *(mx_gu32p)p; }

// 2^(s - 127) as the conversions take it: the byte as a float's exponent (0 means 2^-127 to them)
__device__ __forceinline__ float mx4_scale_f32(uint32_t s) { return __uint_as_float(s << 23); }

// The eight codes of one dword times 2^(s - 127), as bf16 (exact)
__device__ __forceinline__ bf16x8_t mx4_bf16x8(uint32_t w, float scale) {
  u32x4_t v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(bf16x8_t, v);
}

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), b, c, 0, 0, 0);
}

}  // namespace ql
