// Mixture of experts for a few tokens: the router's choice, and the experts' products on MX4 weights.
#include "ql_mx4.hpp"

namespace ql {
namespace {

// ---------------------------------------------------------------- router
// One wave per token.  Logits become unsigned keys of the same order (NaN and -inf become 0, which
// is never taken), lane l holds experts l, 64 + l, ...; each of the k rounds takes the wave's largest
// key and, among the lanes that hold it, the lowest expert.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u || b == 0xFF800000u) return 0u;
  const uint32_t z = b == 0x80000000u ? 0u : b;  // -0 equals 0
  return z ^ ((z >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <int TYPE>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (TYPE == QL_F32) return ((const float*)p)[i];
  else if constexpr (TYPE == QL_BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
  else return (float)((const _Float16*)p)[i];
}

// exp(v - most) where most is the row's largest: 1 at the largest itself, so that rows with
// infinities share their weight among those
__device__ __forceinline__ float weight_of(float v, float most) { return v == most ? 1.0f : expf(v - most); }

template <int TYPE, int NV>
__global__ void __launch_bounds__(256) moe_route_kernel(int64_t T, int E, int k, bool renorm,
                                                        const void* __restrict__ logits, int32_t* __restrict__ ids,
                                                        float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = 64 * i + lane < E ? order_key(load1<TYPE>(logits, t * E + 64 * i + lane)) : 0u;
  uint32_t first = 0, mine = 0;
  float sum = 0.0f;
  int id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = max(top, key[i]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (j == 0) {
      first = top;
      if (!renorm && top) {
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += key[i] ? weight_of(key_value(key[i]), key_value(top)) : 0.0f;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
      }
    }
    if (top == 0u) break;  // nothing left to take
    int e = -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint64_t has = __ballot(key[i] == top);
      if (e < 0 && has) {
        const int l = __builtin_ctzll(has);
        e = 64 * i + l;
        if (lane == l) key[i] = 0u;
      }
    }
    if (lane == j) mine = top, id = e;
    if (renorm) sum += weight_of(key_value(top), key_value(first));
  }
  if (lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = id >= 0 ? weight_of(key_value(mine), key_value(first)) / sum : 0.0f;
  }
}

// ---------------------------------------------------------------- experts
// A pair p = t * k + j is a token and one of its experts.  The workgroups that share an expert find
// its pairs themselves from the ids: which expert is the a-th with any pair, and its pairs in order.
constexpr int kMoeWaves = 8;
constexpr int kMaxPairs = 1024;

struct Picked {
  int expert, pairs;  // expert < 0: fewer than a + 1 experts have pairs
};

// cnt: LDS [E]; list: LDS [kMaxPairs].  All threads call; ends with a barrier.
__device__ Picked find_expert(int a, int P, int E, const int32_t* __restrict__ ids, int* cnt, int* list, int* out) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  if (threadIdx.x == 0) out[0] = -1, out[1] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += blockDim.x) {
    const int e = ids[p];
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int seen = 0, found = -1;
    for (int e0 = 0; e0 < E && found < 0; e0 += 64) {
      const int e = e0 + (int)threadIdx.x;
      const uint64_t has = __ballot(e < E && cnt[e] > 0);
      const int n = __popcll(has);
      if (a < seen + n) {
        const int rank = __popcll(has & ((1ull << threadIdx.x) - 1));
        const uint64_t at = __ballot(((has >> threadIdx.x) & 1) && seen + rank == a);
        found = e0 + __builtin_ctzll(at);
      }
      seen += n;
    }
    if (found >= 0) {
      int n = 0;
      for (int p0 = 0; p0 < P; p0 += 64) {
        const int p = p0 + (int)threadIdx.x;
        const bool is = p < P && ids[p] == found;
        const uint64_t has = __ballot(is);
        if (is) list[n + __popcll(has & ((1ull << threadIdx.x) - 1))] = p;
        n += __popcll(has);
      }
      if (threadIdx.x == 0) out[0] = found, out[1] = n;
    }
  }
  __syncthreads();
  return Picked{out[0], out[1]};
}

// The three bf16 planes of an fp32 value: hi + mid + lo == v to 24 bits (the second product then
// runs on exact bf16 operands); of a value that is not finite only the first is kept.
__device__ __forceinline__ void split3(float v, uint16_t (&h)[3]) {
  h[0] = f32_to_bf16_bits(v);
  const float r = v - bf16_bits_to_f32(h[0]);
  const bool fine = (h[0] & 0x7F80u) != 0x7F80u;
  h[1] = fine ? f32_to_bf16_bits(r) : 0;
  h[2] = fine ? f32_to_bf16_bits(r - bf16_bits_to_f32(h[1])) : 0;
}

// h[p][i] = silu(g) * u with g, u the gate's and the up projection's row i on pair p's token: 16 rows
// of both per workgroup, 16 pairs at a time, the inputs' chunks dealt to the waves.
__global__ void __launch_bounds__(kMoeWaves * 64) moe_gate_up_kernel(int T, int k, int E, int H, int I,
    const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint8_t* __restrict__ gc,
    const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
    uint16_t* __restrict__ h) {
  __shared__ int cnt[QL_MOE_MAX_EXPERTS];
  __shared__ int list[kMaxPairs];
  __shared__ int found[2];
  __shared__ f32x4_t part[kMoeWaves][2][64];
  const int P = T * k;
  const Picked pk = find_expert(blockIdx.y, P, E, ids, cnt, list, found);
  if (pk.expert < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
  const int nblk = H / kMxBlock, nchunk = (nblk + 3) / 4;
  const int n = blockIdx.x * 16 + r;
  const int64_t row = (int64_t)pk.expert * I + (n < I ? n : I - 1), stride = mx4_scale_stride(H);
  for (int p0 = 0; p0 < pk.pairs; p0 += 16) {
    const int slot = p0 + r < pk.pairs ? p0 + r : pk.pairs - 1;
    const uint16_t* xp = x + (int64_t)(list[slot] / k) * H + q * kMxBlock;
    f32x4_t g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
    for (int c = wave; c < nchunk; c += kMoeWaves) {
      const bool in = 4 * c + q < nblk;
      u32x4_t wg = {0u, 0u, 0u, 0u}, wu = wg, a[4] = {};
      float sg = 1.0f, su = 1.0f;
      if (in) {
        wg = ld_b128(gc + row * (H / 2) + c * 64 + q * 16);
        wu = ld_b128(uc + row * (H / 2) + c * 64 + q * 16);
        sg = mx4_scale_f32((ld_b32(gs + row * stride + 4 * c) >> (8 * q)) & 255u);
        su = mx4_scale_f32((ld_b32(us + row * stride + 4 * c) >> (8 * q)) & 255u);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = ld_b128(xp + c * kMxChunk + 8 * j);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g = mfma_bf16(a[j], mx4_bf16x8(wg[j], sg), g);
        u = mfma_bf16(a[j], mx4_bf16x8(wu[j], su), u);
      }
    }
    part[wave][0][lane] = g;
    part[wave][1][lane] = u;
    __syncthreads();
    if (wave == 0) {
      for (int v = 1; v < kMoeWaves; ++v) g += part[v][0][lane], u += part[v][1][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p0 + 4 * q + i < pk.pairs && n < I) {
          uint16_t hv[3];
          split3(g[i] / (1.0f + expf(-g[i])) * u[i], hv);
          const int64_t at = (int64_t)list[p0 + 4 * q + i] * I + n;
#pragma unroll
          for (int z = 0; z < 3; ++z) h[z * (int64_t)P * I + at] = hv[z];
        }
      }
    }
    __syncthreads();
  }
}

// y[t][n] = sum_j w[t][j] (down row n on h[t * k + j]): 16 rows per workgroup, each wave takes whole
// experts in turn and adds to its own token sums in LDS; the waves' sums are joined in wave order.
__global__ void __launch_bounds__(kMoeWaves * 64) moe_down_kernel(int T, int k, int E, int H, int I,
    const uint16_t* __restrict__ h, const int32_t* __restrict__ ids, const float* __restrict__ weights,
    const uint8_t* __restrict__ dc, const uint8_t* __restrict__ ds, float* __restrict__ y) {
  __shared__ int cnt[QL_MOE_MAX_EXPERTS];
  __shared__ float ysum[kMoeWaves][QL_MOE_MAX_TOKENS][16];
  __shared__ int lists[kMoeWaves][kMaxPairs];
  const int P = T * k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  for (int i = lane; i < T * 16; i += 64) ysum[wave][i / 16][i % 16] = 0.0f;
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += blockDim.x) {
    const int e = ids[p];
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  const int nblk = I / kMxBlock, nchunk = (nblk + 3) / 4;
  const int n = blockIdx.x * 16 + r;
  const int64_t stride = mx4_scale_stride(I);
  int* list = lists[wave];
  int seen = 0;
  for (int e = 0; e < E; ++e) {
    if (__builtin_amdgcn_readfirstlane(cnt[e]) == 0) continue;
    if (seen++ % kMoeWaves != wave) continue;
    int pairs = 0;
    for (int p0 = 0; p0 < P; p0 += 64) {
      const int p = p0 + lane;
      const bool is = p < P && ids[p] == e;
      const uint64_t has = __ballot(is);
      if (is) list[pairs + __popcll(has & ((1ull << lane) - 1))] = p;
      pairs += __popcll(has);
    }
    __builtin_amdgcn_wave_barrier();
    const int64_t row = (int64_t)e * H + (n < H ? n : H - 1);
    for (int p0 = 0; p0 < pairs; p0 += 16) {
      const int slot = p0 + r < pairs ? p0 + r : pairs - 1;
      const uint16_t* hp = h + (int64_t)list[slot] * I + q * kMxBlock;
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < nchunk; ++c) {
        const bool in = 4 * c + q < nblk;
        u32x4_t w = {0u, 0u, 0u, 0u}, a[3][4] = {};
        float s = 1.0f;
        if (in) {
          w = ld_b128(dc + row * (I / 2) + c * 64 + q * 16);
          s = mx4_scale_f32((ld_b32(ds + row * stride + 4 * c) >> (8 * q)) & 255u);
#pragma unroll
          for (int z = 0; z < 3; ++z)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[z][j] = ld_b128(hp + z * (int64_t)P * I + c * kMxChunk + 8 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t b = mx4_bf16x8(w[j], s);
#pragma unroll
          for (int z = 0; z < 3; ++z) acc = mfma_bf16(a[z][j], b, acc);
        }
      }
      // one quarter of the wave at a time: a token may hold the same expert twice
      for (int z = 0; z < 4; ++z) {
        if (q == z) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p0 + 4 * q + i < pairs) {
              const int p = list[p0 + 4 * q + i];
              ysum[wave][p / k][r] += weights[p] * acc[i];
            }
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * 16; i += blockDim.x) {
    const int t = i / 16, c = blockIdx.x * 16 + i % 16;
    float s = 0.0f;
    for (int v = 0; v < kMoeWaves; ++v) s += ysum[v][t][i % 16];
    if (c < H) y[(int64_t)t * H + c] = s;
  }
}

template <int TYPE>
void route_as(int64_t T, int E, int k, bool renorm, const void* logits, int32_t* ids, float* weights,
              hipStream_t stream) {
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
  const auto kernel = E <= 64 ? moe_route_kernel<TYPE, 1> : E <= 128 ? moe_route_kernel<TYPE, 2>
                      : E <= 256 ? moe_route_kernel<TYPE, 4> : E <= 512 ? moe_route_kernel<TYPE, 8>
                                                                        : moe_route_kernel<TYPE, 16>;
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, T, E, k, renorm, logits, ids, weights);
}

}  // namespace

hipError_t launch_moe_route(int64_t T, int E, int k, bool renorm, int type, const void* logits, int32_t* ids,
                            float* weights, hipStream_t stream) {
  if (type == QL_F32) route_as<QL_F32>(T, E, k, renorm, logits, ids, weights, stream);
  else if (type == QL_BF16) route_as<QL_BF16>(T, E, k, renorm, logits, ids, weights, stream);
  else route_as<QL_F16>(T, E, k, renorm, logits, ids, weights, stream);
  return hipGetLastError();
}

size_t mx4_moe_workspace_bytes(int64_t T, int64_t k, int64_t I) { return (size_t)(3 * T * k * I * 2); }

hipError_t launch_mx4_moe(const MoeArgs& a, hipStream_t stream) {
  const int P = a.T * a.k, most = P < a.E ? P : a.E;
  uint16_t* h = static_cast<uint16_t*>(a.workspace);
  hipLaunchKernelGGL(moe_gate_up_kernel, dim3((unsigned)((a.I + 15) / 16), (unsigned)most), dim3(kMoeWaves * 64), 0,
                     stream, a.T, a.k, a.E, a.H, a.I, a.x, a.ids, a.gate_codes, a.gate_scales, a.up_codes, a.up_scales,
                     h);
  hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)((a.H + 15) / 16)), dim3(kMoeWaves * 64), 0, stream, a.T, a.k,
                     a.E, a.H, a.I, h, a.ids, a.weights, a.down_codes, a.down_scales, a.y);
  return hipGetLastError();
}

}  // namespace ql
