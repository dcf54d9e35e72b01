// Microscaled 4-bit floats: quantisation, its inverse, and the decode GEMV.
#include "ql_mx4.hpp"

namespace ql {
namespace {

// ---------------------------------------------------------------- quantise
// s = max(0, floor(log2 max|x|) + 127 - 2), so the largest magnitude lands in [4, 8) of the scaled
// block (saturating at 6); codes are x / 2^(s-127) rounded to the nearest e2m1, ties to the even
// code, by the conversion instruction (exact inputs: fp32, and bf16 / fp16 widened).  The exponent
// is the top field of the largest |x| as an integer, which also finds infinities and NaN (255).
// Four lanes share a block: eight inputs each, joined by two lane exchanges, so a wave reads and writes
// whole cache lines.  Bound by memory: 12288 x 4096 in fp32 takes 47 us (4.8 TB/s of the 5.1 that a copy
// reaches), back to fp32 36 us (6.4 TB/s, nearly all of it writes).
template <int TYPE>
__device__ __forceinline__ void load8(const void* W, int64_t i, float (&v)[8]) {
  if constexpr (TYPE == QL_F32) {
    const u32x4_t a = ld_b128_nt((const float*)W + i), b = ld_b128_nt((const float*)W + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(a[j]), v[4 + j] = __uint_as_float(b[j]);
  } else {
    const u32x4_t a = ld_b128_nt((const uint16_t*)W + i);
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
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true));  // lane ^ 1
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true));  // lane ^ 2
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
// y[m][n] = sum_k W[n][k] x[m][k]: a workgroup owns R tiles of 16 rows and one of the gridDim.y parts
// of the inputs, its waves take pairs of chunks in turn and their sums are joined through LDS in wave
// order; parts (more than one) go to `out` = [part][M][N] for mx4_join_kernel.  Bound by the stream of
// W and the tokens that go with it: weights from HBM, in us (and TB/s of W) at one token 4096 x 4096 4.3
// (2.1), 12288 x 4096 7.5 (3.5), 5120 x 17408 14.4 (3.3), at 16 tokens 28672 x 8192 36 (3.5); about 2 us of
// each is the launch.
constexpr int kGemvWaves = 8;

template <int R, int XP, bool TAIL>
__global__ void __launch_bounds__(kGemvWaves * 64) mx4_gemv_kernel(int M, int N, int K,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const uint16_t* __restrict__ x,
    float* __restrict__ out) {
  constexpr int WAVES = kGemvWaves;
  using S = Skinny<1, R, XP>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WAVES * S::kLds];
  static_assert(S::kLds >= R * 1024, "the sums are joined in the same memory");
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
  const int last = (int)min((int64_t)16 * R, N - n0) - 1;  // rows past N repeat the last one, tokens past M too
  S job;
  const uint8_t* const c[1] = {codes + n0 * (K / 2)};
  const uint8_t* const s[1] = {scales + n0 * mx4_scale_stride(K)};
  f32x4_t acc[1][R];
  bool once = true;
  job.template run<TAIL>(
      smem + wave * S::kLds, K, (int)blockIdx.y * WAVES + wave, WAVES * (int)gridDim.y, r < 2 * XP ? r : 0, 1,
      [&](S& j) {
        if (once) j.init(K, c, s, [&](int t, int i) { return min(16 * t + i, last); }, x, [&](int m) { return min(m, M - 1); });
        const bool is = once;
        once = false;
        return is;
      },
      [&](const f32x4_t(&sums)[1][R]) {
#pragma unroll
        for (int t = 0; t < R; ++t) acc[0][t] = sums[0][t];
      });
  __syncthreads();
  f32x4_t* part = reinterpret_cast<f32x4_t*>(smem);
#pragma unroll
  for (int t = 0; t < R; ++t) part[(wave * R + t) * 64 + lane] = acc[0][t];
  __syncthreads();
  out += (int64_t)blockIdx.y * M * N;
  for (int t = wave; t < R; t += WAVES) {
    f32x4_t v = part[t * 64 + lane];
    for (int u = 1; u < WAVES; ++u) v += part[(u * R + t) * 64 + lane];
    const int64_t n = n0 + 16 * t + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * q + i < M && n < N) out[(int64_t)(4 * q + i) * N + n] = v[i];
  }
}

template <int R, int XP>
hipError_t gemv_as(int M, int N, int K, const uint8_t* codes, const uint8_t* scales, const uint16_t* x, int parts,
                   float* out, hipStream_t stream) {
  const auto kernel = K % (2 * kMxChunk) ? mx4_gemv_kernel<R, XP, true> : mx4_gemv_kernel<R, XP, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((N + 16 * R - 1) / (16 * R)), (unsigned)parts), dim3(kGemvWaves * 64), 0, stream,
                     M, N, K, codes, scales, x, out);
  return hipGetLastError();
}

template <int XP>
hipError_t gemv_tokens(const GemvPlan& g, int M, int N, int K, const uint8_t* codes, const uint8_t* scales,
                       const uint16_t* x, float* out, hipStream_t stream) {
  if (g.tiles == 4) return gemv_as<4, XP>(M, N, K, codes, scales, x, g.parts, out, stream);
  if (g.tiles == 2) return gemv_as<2, XP>(M, N, K, codes, scales, x, g.parts, out, stream);
  return gemv_as<1, XP>(M, N, K, codes, scales, x, g.parts, out, stream);
}

// y = the sum of `parts` arrays of n floats, in order
__global__ void __launch_bounds__(256) mx4_join_kernel(int64_t n, int parts, const float* __restrict__ in,
                                                       float* __restrict__ y) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float v = in[i];
    for (int p = 1; p < parts; ++p) v += in[p * n + i];
    y[i] = v;
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

hipError_t launch_mx4_join(int64_t n, int parts, const float* in, float* y, hipStream_t stream) {
  const int64_t want = (n + 255) / 256, most = 8 * (int64_t)device_cu_count();
  hipLaunchKernelGGL(mx4_join_kernel, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, stream, n, parts, in, y);
  return hipGetLastError();
}

// What a CU has to fetch decides: a workgroup reads 17/32 bytes of each weight of its 16 R rows and
// token_bytes per input, the tokens over again for every workgroup.  Few rows leave CUs
// idle, so the rows per workgroup and the parts of K are chosen together for the least bytes per CU;
// a second launch to join parts costs about 5 us, 175 KB at the 35 KB/us that a CU was seen to fetch
// whatever the number of its waves (5120 x 17408 at 16 tokens: 28 / 22 / 29 us with 1 / 2 / 4 tiles, 18.0 with
// 4 tiles and three parts; 4096 x 14336 at 8: 12.2 with 1 tile, 14.3 with 4 and three parts).
GemvPlan mx4_stream_plan(double token_bytes, int N, int K) {
  const int64_t cus = device_cu_count(), pairs = (K + 2 * kMxChunk - 1) / (2 * kMxChunk);
  GemvPlan best{1, 1};
  double least = 0.0;
  for (int tiles = 1; tiles <= 4; tiles *= 2)
    for (int parts = 1; parts <= 8 && (parts == 1 || pairs >= 8 * parts); ++parts) {
      const int64_t groups = ((int64_t)N + 16 * tiles - 1) / (16 * tiles) * parts;
      const double rounds = (double)((groups + cus - 1) / cus);
      const double cost = rounds * (8.5 * tiles + token_bytes) * K / parts + (parts > 1 ? 175e3 : 0.0);
      if (least == 0.0 || cost < least) least = cost, best = {tiles, parts};
    }
  return best;
}

GemvPlan mx4_gemv_plan(int M, int N, int K) {
  return mx4_stream_plan(M <= 2 ? 4.0 : M <= 4 ? 8.0 : M <= 8 ? 16.0 : 32.0, N, K);
}

hipError_t launch_mx4_gemv(const GemvPlan& g, int M, int N, int K, const uint8_t* codes, const uint8_t* scales,
                           const uint16_t* x, float* y, float* workspace, hipStream_t stream) {
  float* out = g.parts > 1 ? workspace : y;
  const hipError_t e = M <= 2   ? gemv_tokens<1>(g, M, N, K, codes, scales, x, out, stream)
                       : M <= 4 ? gemv_tokens<2>(g, M, N, K, codes, scales, x, out, stream)
                       : M <= 8 ? gemv_tokens<4>(g, M, N, K, codes, scales, x, out, stream)
                                : gemv_tokens<8>(g, M, N, K, codes, scales, x, out, stream);
  if (e != hipSuccess || g.parts == 1) return e;
  return launch_mx4_join((int64_t)M * N, g.parts, workspace, y, stream);
}

}  // namespace ql
