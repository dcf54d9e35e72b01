// Rotary positions: the heads of q and k, optionally normed, are turned by their token's position; q goes out
// as bf16, k and v into the paged cache.
#include "ql_attn.hpp"

namespace ql {
namespace {

template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (TYPE == QL_F32) {
    typedef const __attribute__((address_space(1))) at_f32x4* f4p;
    const at_f32x4 a = ((f4p)((const float*)p + at))[0], b = ((f4p)((const float*)p + at))[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  } else {
    const u32x4_t w = *(gu32x4p)((const uint16_t*)p + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == QL_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i]);
        x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
      }
    }
  }
}

// the nearest e4m3 values, what is over 448 as 448, NaN as NaN
__device__ __forceinline__ float into_e4m3(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(into_e4m3(a), into_e4m3(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(into_e4m3(c), into_e4m3(d), w, true);
}

__device__ __forceinline__ u32x4_t bf16x8(const float (&x)[8]) {
  return u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}

// A workgroup takes one token and up to 2048 / D of its heads (q, then k, then v), eight dims a lane.  The
// token's cosines and sines are made once, by the first R / 2 lanes, while the heads' loads are under way: the
// angle in turns as a 64-bit product (a 32-bit one is off by a radian at position 2^24), its fraction in fp32.  A
// pair's other half is in another lane: heads meet in LDS.
//
// Memory bounds: 8192 tokens of 40 + 2 x 8 heads of 128 (346 MB, fp32 in, bf16 out) take 67 us, 5.1 TB/s, where a
// large copy reaches 4.9.  bf16 or fp16 in (231 MB) takes 61, 3.8 TB/s, without norms 54: there the waves' own time counts
// too (norms' sums over lanes, sines, the pairs' way through LDS).  e4m3 pages, a division a value, cost 2 to 3 us
// more for 16 MB less.  One token is a launch and two memory latencies, 3.8 us.
template <int TYPE, int D, bool F8>
__global__ void __launch_bounds__(256) rope_append_kernel(RopeArgs a) {
  constexpr int LANES = D / 8, HEADS = 256 / LANES;
  __shared__ float cs[D / 2][2];
  __shared__ __attribute__((aligned(16))) float xs[HEADS][D + 4];
  const int t = blockIdx.x, slot_in = threadIdx.x / LANES, part = threadIdx.x % LANES;
  const int h = blockIdx.y * HEADS + slot_in, Hkv = a.kv.heads;
  const bool live = h < a.Hq + 2 * Hkv, is_q = h < a.Hq, is_k = !is_q && h < a.Hq + Hkv;
  const int hk = is_q ? h : is_k ? h - a.Hq : h - a.Hq - Hkv;  // of its own tensor
  float x[8] = {};
  if (live) {
    const void* p = is_q ? a.q : is_k ? a.k : a.v;
    const int64_t stride = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
    load8<TYPE>(p, t * stride + hk * D + part * 8, x);
  }
  const int half = a.dims / 2;
  if ((int)threadIdx.x < half) {
    const double turns = (double)a.positions[t] * (double)a.freqs[threadIdx.x] * 0.15915494309189533577;
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[threadIdx.x][0] = c * a.factor, cs[threadIdx.x][1] = s * a.factor;
  }
  const float* norm = is_q ? a.q_norm : a.k_norm;
  if (norm && (is_q || is_k)) {
    float by[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) by[i] = norm[part * 8 + i];
    auto squares = [&] {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
#pragma unroll
      for (int m = 1; m < LANES; m *= 2) sum += __shfl_xor(sum, m);
      return sum;
    };
    const float mean = squares() * (1.0f / D) + a.eps;
    float r = 1.0f / sqrtf(mean);
    if (__builtin_expect(!(mean < 0x1p119f && mean > 0x1p-100f), 0)) {
      // fp32 may not hold the squares: those of x times a power of two, which cancels out
      const float f = mean < 1.0f ? 0x1p100f : 0x1p-70f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= f;
      r = 1.0f / sqrtf(squares() * (1.0f / D) + a.eps * f * f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * by[i];
  }
  {
    at_f32x4* at = (at_f32x4*)&xs[slot_in][part * 8];
    at[0] = at_f32x4{x[0], x[1], x[2], x[3]};
    at[1] = at_f32x4{x[4], x[5], x[6], x[7]};
  }
  __syncthreads();
  if (!live) return;
  if (is_q || is_k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = part * 8 + i;
      if (d < a.dims) {
        const bool second = a.interleaved ? i & 1 : d >= half;
        const int pair = a.interleaved ? d >> 1 : second ? d - half : d;
        const int other = a.interleaved ? d ^ 1 : second ? d - half : d + half;
        const float c = cs[pair][0], s = cs[pair][1];
        x[i] = x[i] * c + xs[slot_in][other] * (second ? s : -s);
      }
    }
  }
  if (is_q) {
    *(u32x4_t*)(a.out + ((int64_t)t * a.Hq + h) * D + part * 8) = bf16x8(x);
    return;
  }
  const int slot = a.slots[t];
  if (slot < 0 || slot >> a.kv.page_shift >= a.kv.pages) return;
  const int64_t page = slot >> a.kv.page_shift, in = slot & ((1 << a.kv.page_shift) - 1);
  const int64_t at = (((page * Hkv + hk) << a.kv.page_shift) + in) * D + part * 8;
  uint8_t* cache = is_k ? a.kv.k : a.kv.v;
  if constexpr (F8) {
    const float s = (is_k ? a.kv.k_scale : a.kv.v_scale)[hk];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] /= s;
    *(u32x2_t*)(cache + at) = u32x2_t{e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7])};
  } else {
    *(u32x4_t*)(cache + 2 * at) = bf16x8(x);
  }
}

template <int TYPE, int D>
void launch(const RopeArgs& a, hipStream_t stream) {
  constexpr int HEADS = 2048 / D;
  const dim3 grid(a.T, (a.Hq + 2 * a.kv.heads + HEADS - 1) / HEADS);
  if (a.kv.f8) rope_append_kernel<TYPE, D, true><<<grid, 256, 0, stream>>>(a);
  else rope_append_kernel<TYPE, D, false><<<grid, 256, 0, stream>>>(a);
}
template <int TYPE>
void launch_dim(const RopeArgs& a, hipStream_t stream) {
  if (a.kv.dim == 64) launch<TYPE, 64>(a, stream);
  else launch<TYPE, 128>(a, stream);
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t stream) {
  if (a.dtype == QL_F32) launch_dim<QL_F32>(a, stream);
  else if (a.dtype == QL_BF16) launch_dim<QL_BF16>(a, stream);
  else launch_dim<QL_F16>(a, stream);
  return hipGetLastError();
}

}  // namespace ql
