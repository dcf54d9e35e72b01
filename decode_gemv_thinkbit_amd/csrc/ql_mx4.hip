// Microscaled 4-bit floats: quantisation, its inverse, and the decode GEMV.
#include "ql_mx4.hpp"

namespace ql {
namespace {

// ---------------------------------------------------------------- quantise
// s = max(0, floor(log2 max|x|) + 127 - 2), so the largest magnitude lands in [4, 8) of the scaled
// block (saturating at 6); codes are x / 2^(s-127) rounded to the nearest e2m1, ties to the even
// code, by the conversion instruction (exact inputs: fp32, and bf16 / fp16 widened).  The exponent
// is the top field of the largest |x| as an integer, which also finds infinities and NaN (255).
// Four lanes share a block: eight inputs each, joined by two lane exchanges.
template <int TYPE>
__device__ __forceinline__ void load8(const void* W, int64_t i, float (&v)[8]) {
  if constexpr (TYPE == QL_F32) {
    const u32x4_t a = ld_b128((const float*)W + i), b = ld_b128((const float*)W + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(a[j]), v[4 + j] = __uint_as_float(b[j]);
  } else {
    const u32x4_t a = ld_b128((const uint16_t*)W + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == QL_BF16) {
        v[2 * j] = __uint_as_float(a[j] << 16);
        v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
      } else {
        v[2 * j] = (float)__builtin_bit_cast(_Float16, (uint16_t)a[j]);
        v[2 * j + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(a[j] >> 16));
      }
    }
  }
}

// Element i of a row-major [rows][K] matrix sits at i (K % 32 == 0), so lanes run over groups of
// eight elements without regard to rows; only the scale rows, padded to whole dwords, need the row.
// `block` is below 2^31 (the callers bound the element count by 2^36).
__device__ __forceinline__ int64_t scale_index(uint32_t block, uint32_t nblk, uint32_t stride) {
  return stride == nblk ? (int64_t)block : (int64_t)(block / nblk) * stride + block % nblk;
}

template <int TYPE>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(int64_t groups, uint32_t nblk, uint32_t stride,
                                                           const void* __restrict__ W, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  // groups is a multiple of four, and so is every grid step: a block's four lanes run together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups; i += (int64_t)gridDim.x * 256) {
    float v[8];
    load8<TYPE>(W, i * 8, v);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t e = top >> 23;
    const uint32_t s = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
    const float scale = mx4_scale_f32(s);
    uint32_t w = 0;
    if (s != 255u) {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
    }
    reinterpret_cast<uint32_t*>(codes)[i] = w;
    if ((i & 3) == 0) {
      const uint32_t b = (uint32_t)(i >> 2);
      const int64_t at = scale_index(b, nblk, stride);
      scales[at] = (uint8_t)s;
      if (stride != nblk && b % nblk == nblk - 1)  // the row's padding
        for (uint32_t p = 1; p <= stride - nblk; ++p) scales[at + p] = 0;
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(256) mx4_dequant_kernel(int64_t groups, uint32_t nblk, uint32_t stride,
                                                          const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, void* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups; i += (int64_t)gridDim.x * 256) {
    const uint32_t w = ld_b32(codes + i * 4);
    const float scale = mx4_scale_f32(scales[scale_index((uint32_t)(i >> 2), nblk, stride)]);
    if constexpr (BF16) {
      reinterpret_cast<u32x4_t*>(out)[i] = __builtin_bit_cast(u32x4_t, mx4_bf16x8(w, scale));
    } else {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
      const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
      const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
      f32x4_t* p = reinterpret_cast<f32x4_t*>(out) + 2 * i;
      p[0] = f32x4_t{a[0], a[1], b[0], b[1]};
      p[1] = f32x4_t{c[0], c[1], d[0], d[1]};
    }
  }
}

// ---------------------------------------------------------------- decode GEMV
// y[m][n] = sum_k W[n][k] x[m][k]: a workgroup owns 16 rows, its waves take chunks in turn and
// their sums are joined through LDS in wave order.
constexpr int kGemvWaves = 8;

__global__ void __launch_bounds__(kGemvWaves * 64) mx4_gemv_kernel(int M, int N, int K,
                                                                  const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  const uint16_t* __restrict__ x,
                                                                  float* __restrict__ y) {
  __shared__ f32x4_t part[kGemvWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
  const int nblk = K / kMxBlock, nchunk = (nblk + 3) / 4;
  const int64_t n = (int64_t)blockIdx.x * 16 + r, row = n < N ? n : N - 1;  // rows past N repeat the last one
  const uint8_t* wp = codes + row * (K / 2) + q * 16;
  const uint8_t* sp = scales + row * mx4_scale_stride(K);
  const uint16_t* xp = x + (int64_t)(r < M ? r : M - 1) * K + q * kMxBlock;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = wave; c < nchunk; c += kGemvWaves) {
    const bool in = 4 * c + q < nblk;  // blocks past K are zeros on both sides
    u32x4_t w = {0u, 0u, 0u, 0u}, a[4] = {};
    float s = 1.0f;
    if (in) {
      w = ld_b128(wp + c * 64);
      s = mx4_scale_f32((ld_b32(sp + 4 * c) >> (8 * q)) & 255u);
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = ld_b128(xp + c * kMxChunk + 8 * j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = mfma_bf16(a[j], mx4_bf16x8(w[j], s), acc);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    for (int v = 1; v < kGemvWaves; ++v) acc += part[v][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * q + i < M && n < N) y[(int64_t)(4 * q + i) * N + n] = acc[i];
  }
}

}  // namespace

// eight elements per lane, at most eight workgroups a CU
static dim3 stream_grid(int64_t groups) {
  const int64_t want = (groups + 255) / 256, most = 8 * (int64_t)device_cu_count();
  return dim3((unsigned)(want < most ? want : most));
}

hipError_t launch_mx4_quantize(int64_t rows, int64_t K, int type, const void* W, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream) {
  const int64_t groups = rows * (K / 8);
  const auto kernel = type == QL_F32 ? mx4_quantize_kernel<QL_F32>
                      : type == QL_BF16 ? mx4_quantize_kernel<QL_BF16> : mx4_quantize_kernel<QL_F16>;
  hipLaunchKernelGGL(kernel, stream_grid(groups), dim3(256), 0, stream, groups, (uint32_t)(K / kMxBlock),
                     (uint32_t)mx4_scale_stride(K), W, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales, bool bf16,
                              void* out, hipStream_t stream) {
  const int64_t groups = rows * (K / 8);
  const auto kernel = bf16 ? mx4_dequant_kernel<true> : mx4_dequant_kernel<false>;
  hipLaunchKernelGGL(kernel, stream_grid(groups), dim3(256), 0, stream, groups, (uint32_t)(K / kMxBlock),
                     (uint32_t)mx4_scale_stride(K), codes, scales, out);
  return hipGetLastError();
}

hipError_t launch_mx4_gemv(int M, int N, int K, const uint8_t* codes, const uint8_t* scales, const uint16_t* x,
                           float* y, hipStream_t stream) {
  hipLaunchKernelGGL(mx4_gemv_kernel, dim3((unsigned)((N + 15) / 16)), dim3(kGemvWaves * 64), 0, stream, M, N, K,
                     codes, scales, x, y);
  return hipGetLastError();
}

}  // namespace ql
