// MX4 x MX4 GEMM: both operands are read as stored by the scaled matrix instruction.
#include "ql_mx4.hpp"

namespace ql {
namespace {

// y[m][n] = sum_k X[m][k] W[n][k].  128 x 128 outputs per workgroup, 64 x 64 per wave as two by two
// v_mfma_scale_f32_32x32x64: lane l holds row l % 32, block l / 32 of a 64-input step.
__global__ void __launch_bounds__(256) mx4_gemm_kernel(int M, int N, int K, const uint8_t* __restrict__ xc,
                                                       const uint8_t* __restrict__ xs, const uint8_t* __restrict__ wc,
                                                       const uint8_t* __restrict__ ws, float* __restrict__ y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5, r = lane & 31;
  const int64_t m0 = (int64_t)blockIdx.y * 128 + (wave >> 1) * 64, n0 = (int64_t)blockIdx.x * 128 + (wave & 1) * 64;
  const int nblk = K / kMxBlock, nchunk = (nblk + 3) / 4;
  const int64_t stride = mx4_scale_stride(K);
  const uint8_t *ap[2], *as[2], *bp[2], *bs[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {  // rows past the end repeat the last one
    const int64_t m = m0 + 32 * t + r < M ? m0 + 32 * t + r : M - 1, n = n0 + 32 * t + r < N ? n0 + 32 * t + r : N - 1;
    ap[t] = xc + m * (K / 2), as[t] = xs + m * stride;
    bp[t] = wc + n * (K / 2), bs[t] = ws + n * stride;
  }
  f32x16_t acc[2][2] = {};
  for (int c = 0; c < nchunk; ++c) {
    uint32_t sa[2], sb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) sa[t] = ld_b32(as[t] + 4 * c), sb[t] = ld_b32(bs[t] + 4 * c);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int q = 2 * st + half, b = 4 * c + q;
      const bool in = b < nblk;
      i32x8_t A[2], B[2];
      int fa[2], fb[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4_t a = {0u, 0u, 0u, 0u}, w = {0u, 0u, 0u, 0u};
        if (in) a = ld_b128(ap[t] + b * 16), w = ld_b128(bp[t] + b * 16);
        A[t] = i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
        B[t] = i32x8_t{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
        fa[t] = in ? (int)((sa[t] >> (8 * q)) & 255u) : 127;
        fb[t] = in ? (int)((sb[t] >> (8 * q)) & 255u) : 127;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A[i], B[j], acc[i][j], 4, 4, 0, fa[i], 0, fb[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t m = m0 + 32 * i + (v >> 2) * 8 + half * 4 + (v & 3), n = n0 + 32 * j + r;
        if (m < M && n < N) y[m * N + n] = acc[i][j][v];
      }
}

}  // namespace

hipError_t launch_mx4_gemm(int M, int N, int K, const uint8_t* xc, const uint8_t* xs, const uint8_t* wc,
                           const uint8_t* ws, float* y, hipStream_t stream) {
  hipLaunchKernelGGL(mx4_gemm_kernel, dim3((unsigned)((N + 127) / 128), (unsigned)((M + 127) / 128)), dim3(256), 0,
                     stream, M, N, K, xc, xs, wc, ws, y);
  return hipGetLastError();
}

}  // namespace ql
