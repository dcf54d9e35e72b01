// Rotary positions, the paged key-value cache and attention over it: launchers, and what their kernels share.
//
// The cache is k, v [pages][heads][page][D]: a page's tokens of one kv head lie together (page * D values),
// so whoever reads a head streams whole pages.  Values are bf16, or e4m3 times one fp32 scale per head, which
// is multiplied into the scores (keys) and the output (values), never into the cached numbers.
#pragma once

#include "ql_internal.hpp"
#include "ql_stream.hpp"

namespace ql {

struct KvArgs {
  uint8_t *k, *v;
  const float *k_scale, *v_scale;  // per head, or null
  int32_t pages, heads, page_shift, dim;
  bool f8;
};

struct RopeArgs {
  KvArgs kv;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t *positions, *slots;
  const float *freqs, *q_norm, *k_norm;
  uint16_t* out;
  float factor, eps;
  int32_t T, Hq, dims, dtype;
  bool interleaved;
};
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t stream);

struct AttnArgs {
  KvArgs kv;
  const uint16_t* q;
  const int32_t *starts, *table, *lens;  // starts: prompts only
  int64_t table_stride;
  uint16_t* out;
  float* ws;
  float score_scale;  // scale * log2(e)
  int32_t T, B, Hq, keys;  // keys: the most a row of the table holds
};
size_t attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys);
hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream);
size_t attn_prompt_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys);
int64_t attn_prompt_blocks(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys);
hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- device helpers
typedef __attribute__((ext_vector_type(8))) __bf16 at_bf16x8;
typedef __attribute__((ext_vector_type(4))) float at_f32x4;
typedef __attribute__((ext_vector_type(16))) float at_f32x16;

constexpr float kNegInf = -__builtin_inff();
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Weights are exp2(score - maximum - room), the maximum in use being `lag` below a score at most, so that those of a
// sequence's len tokens sum to 1/2 at most and times the largest values stay in fp32's range.  The room is no larger than
// that, as at the other end of the range values lose what it takes (with room for 2^30 tokens, V of 2^-112 came out
// as 0 for one).  It is one for all parts of a row, so it cancels out; up to 40 as it is, it puts a weight's exponent off by
// 2^-19, where a bf16 weight is off by 2^-8.
__device__ __forceinline__ float room_of(int len, float lag) { return lag + (float)(33 - __builtin_clz(len | 1)); }

// what a call reads once: not kept in the caches
template <class P>
__device__ __forceinline__ auto load_once(P p) { return __builtin_nontemporal_load(p); }

// two fp32 as a dword of bf16, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf2;
  typedef __attribute__((ext_vector_type(2))) float f2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), bf2));
}

// four e4m3 values as two dwords of bf16 (exact)
__device__ __forceinline__ u32x2_t bf16_of_e4m3(uint32_t w) {
  return u32x2_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
}

// The largest of the lanes l, l ^ 32 (and, with 16, of all four with the same l % 16), in each of them
__device__ __forceinline__ float max_xor32(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float max_xor16(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_xor32(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float sum_xor16(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// What a part with maximum m weighs in a sum whose maximum is `most` (equal infinities: 1, as m - most is NaN)
__device__ __forceinline__ float part_weight(float m, float most) { return m == most ? 1.0f : exp2_fast(m - most); }

// the sum over the lanes up to this one, and the whole wave's in every lane
__device__ __forceinline__ uint32_t scan_lanes(uint32_t v) {
  auto from = [](uint32_t x, auto ctrl, auto rows) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  using std::integral_constant;
  v += from(v, integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  v += from(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});
  return v + from(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }

}  // namespace ql
