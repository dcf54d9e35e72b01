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

// Lane 63 gathers the wave by row shifts and row broadcasts (a tenth of the latency of six LDS exchanges).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lanes_of(uint32_t v) {  // 0 where no lane is read
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, lanes_of<0x111, 0xF>(v));
  v = max(v, lanes_of<0x112, 0xF>(v));
  v = max(v, lanes_of<0x114, 0xF>(v));
  v = max(v, lanes_of<0x118, 0xF>(v));
  v = max(v, lanes_of<0x142, 0xA>(v));
  v = max(v, lanes_of<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float f) {
  auto step = [&](uint32_t other) { f += __uint_as_float(other); };
  step(lanes_of<0x111, 0xF>(__float_as_uint(f)));
  step(lanes_of<0x112, 0xF>(__float_as_uint(f)));
  step(lanes_of<0x114, 0xF>(__float_as_uint(f)));
  step(lanes_of<0x118, 0xF>(__float_as_uint(f)));
  step(lanes_of<0x142, 0xA>(__float_as_uint(f)));
  step(lanes_of<0x143, 0xC>(__float_as_uint(f)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), 63));
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
    top = wave_max(top);
    if (j == 0) {
      first = top;
      if (!renorm && top) {
#pragma unroll
        for (int i = 0; i < NV; ++i) sum += key[i] ? weight_of(key_value(key[i]), key_value(top)) : 0.0f;
        sum = wave_sum(sum);
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
// A pair p = t * k + j is a token and one of its experts.  An expert's pairs, in order, make groups of up
// to G, which share a read of its matrices.  Every workgroup finds them itself from the ids, into LDS: up
// to 64 pairs in registers, every wave for itself; more by counting, with four barriers.
constexpr int kMaxPairs = QL_MOE_MAX_TOKENS * QL_MOE_MAX_TOPK;
constexpr int kFewPairs = 256;  // three workgroups of the gate and up kernel fit a CU's LDS, not two

template <int PAIRS, int G, bool WEIGHTS>  // PAIRS: 64, or the most there may be
struct Groups {
  static constexpr bool SMALL = PAIRS == 64;
  static constexpr int kSlots = SMALL ? 64 * G : PAIRS;
  struct Storage {
    uint32_t group[PAIRS];               // expert, pairs << 10, first slot << 16
    uint32_t pair[kSlots];                   // pair, token << 16
    float weight[WEIGHTS ? kSlots : 1];      // its weight
    int groups;
  };
  struct Scratch {  // while finding (SMALL: not used); afterwards the memory is the caller's again
    uint32_t count[QL_MOE_MAX_EXPERTS], start[QL_MOE_MAX_EXPERTS];
    uint16_t id[kMaxPairs], rank[kMaxPairs];
  };

  // the lanes that hold the same id (0 for a lane without one), by its bits
  static __device__ __forceinline__ uint64_t same(int id, bool is, int E) {
    uint64_t like = __ballot(is);
    for (int b = 0; (1 << b) < E; ++b) {
      const uint64_t ones = __ballot((id >> b) & 1);
      like &= (id >> b) & 1 ? ones : ~ones;
    }
    return is ? like : 0;
  }
  // All threads; returns the number of groups.  weights: of the pairs (WEIGHTS).
  static __device__ int find(int P, int E, int k, const int32_t* __restrict__ ids, const float* __restrict__ weights,
                             Storage& st, uint8_t* scratch) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t below = (1ull << lane) - 1;
    if constexpr (SMALL) {
      const int raw = lane < P ? ids[lane] : -1, id = raw < E ? raw : -1;  // negative: none
      const float w = WEIGHTS && lane < P ? weights[lane] : 0.0f;
      const uint64_t like = same(id, id >= 0, E);
      const int rank = __popcll(like & below), r0 = rank - rank % G;
      uint64_t from = like;  // the group's pairs and those behind it
      for (int i = 0; i < r0; ++i) from &= from - 1;
      const int lead = from ? __builtin_ctzll(from) : 0, size = min(G, (int)__popcll(from));
      const uint64_t firsts = __ballot(id >= 0 && rank == r0);
      const int group = __popcll(firsts & ((1ull << lead) - 1));
      if (id >= 0) {
        st.pair[group * G + rank % G] = (uint32_t)lane | (uint32_t)(lane / k) << 16;
        if (WEIGHTS) st.weight[group * G + rank % G] = w;
        if (rank % G == 0) st.group[group] = (uint32_t)id | (uint32_t)size << 10 | (uint32_t)(group * G) << 16;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every wave reads what it wrote
      return __popcll(firsts);
    } else {
      Scratch& sc = *reinterpret_cast<Scratch*>(scratch);
      for (int e = threadIdx.x; e < E; e += blockDim.x) sc.count[e] = 0u;
      for (int p0 = wave * 64; p0 < P; p0 += (int)blockDim.x) {  // places among the 64 pairs around
        const int p = p0 + lane, raw = p < P ? ids[p] : -1, e = raw >= 0 && raw < E ? raw : 65535;
        const int before = (int)__popcll(same(e, e != 65535, E) & below);
        if (p < P) sc.id[p] = (uint16_t)e, sc.rank[p] = (uint16_t)before;
      }
      __syncthreads();
      if (wave == 0) {
        for (int p0 = 0; p0 < P; p0 += 64) {  // places among all, 64 after 64
          const int p = p0 + lane, e = p < P ? sc.id[p] : 65535;
          if (e != 65535) {
            sc.rank[p] = (uint16_t)(sc.rank[p] + sc.count[e]);
            atomicAdd(&sc.count[e], 1u);
          }
        }
        int slots = 0, groups = 0;  // running totals over the experts
        for (int e0 = 0; e0 < E; e0 += 64) {
          const int n = e0 + lane < E ? (int)sc.count[e0 + lane] : 0;
          int both = n | ((n + G - 1) / G) << 16;
          for (int d = 1; d < 64; d *= 2) {
            const int left = __shfl_up(both, d);
            if (lane >= d) both += left;
          }
          if (e0 + lane < E) {
            const int before = both - (n | ((n + G - 1) / G) << 16);
            sc.start[e0 + lane] = (uint32_t)(slots + (before & 0xFFFF)) | (uint32_t)(groups + (before >> 16)) << 16;
          }
          const int all = __shfl(both, 63);
          slots += all & 0xFFFF, groups += all >> 16;
        }
        if (lane == 0) st.groups = groups;
      }
      __syncthreads();
      for (int p = threadIdx.x; p < P; p += blockDim.x) {
        const int e = sc.id[p], rank = sc.rank[p];
        if (e == 65535) continue;
        const int slot = (int)(sc.start[e] & 0xFFFF) + rank, group = (int)(sc.start[e] >> 16) + rank / G;
        st.pair[slot] = (uint32_t)p | (uint32_t)(p / k) << 16;
        if (WEIGHTS) st.weight[slot] = weights[p];
        if (rank % G == 0)
          st.group[group] = (uint32_t)e | (uint32_t)min(G, (int)sc.count[e] - rank) << 10 | (uint32_t)slot << 16;
      }
      __syncthreads();
      return __builtin_amdgcn_readfirstlane(st.groups);
    }
  }
};

// a group's record, uniform
struct Group {
  int expert, count, first;
  __device__ __forceinline__ explicit Group(uint32_t record) {
    const uint32_t v = __builtin_amdgcn_readfirstlane(record);
    expert = (int)(v & 1023u), count = (int)((v >> 10) & 63u), first = (int)(v >> 16);
  }
};

// The three bf16 planes of an fp32 value: hi + mid + lo == v to 24 bits (the second product then
// runs on exact bf16 operands); of a value that is not finite only the first is kept.
__device__ __forceinline__ void split3(float v, uint16_t (&h)[3]) {
  h[0] = f32_to_bf16_bits(v);
  const float r = v - bf16_bits_to_f32(h[0]);
  const bool fine = (h[0] & 0x7F80u) != 0x7F80u;
  h[1] = fine ? f32_to_bf16_bits(r) : 0;
  h[2] = fine ? f32_to_bf16_bits(r - bf16_bits_to_f32(h[1])) : 0;
}

// h[p][i] = silu(g) * u with g, u the gate's and the up projection's row i on pair p's token.  A task is 16
// rows of both for one group.  JOIN (few tasks): workgroups take tasks in turn, the inputs' pairs of
// chunks dealt to the four waves and their sums joined in wave order; else every wave takes tasks of its
// own.  Either way the next task's loads are under way while one ends.
template <int XP, bool JOIN, bool SMALL, bool TAIL>
__global__ void __launch_bounds__(256) moe_gate_up_kernel(int T, int k, int E, int H, int I,
    const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint8_t* __restrict__ gc,
    const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
    uint16_t* __restrict__ h, uint32_t* __restrict__ counters, int ncounters) {
  constexpr int G = 2 * XP, kPairs = SMALL ? 64 : XP == 2 ? kFewPairs : kMaxPairs;
  using S = Skinny<2, 1, XP, 2>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * S::kLds];
  __shared__ typename Groups<kPairs, G, false>::Storage plan;
  __shared__ f32x4_t part[JOIN ? 2 : 1][JOIN ? 4 : 1][2][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, r = lane & 15;
  const int P = T * k, tiles = (I + 15) / 16;
  // the second kernel's counters start at zero
  for (int i = blockIdx.x * 256 + threadIdx.x; i < ncounters; i += gridDim.x * 256) counters[i] = 0u;
  const int tasks = Groups<kPairs, G, false>::find(P, E, k, ids, nullptr, plan, smem) * tiles;
  const int first = JOIN ? (int)blockIdx.x : 4 * (int)blockIdx.x + wave, step = (JOIN ? 1 : 4) * (int)gridDim.x;
  const int mine = tasks > first ? (tasks - 1 - first) / step + 1 : 0;
  S job;
  int ahead = first, now = first;
  auto finish = [&](float g, float u, int slot) __attribute__((always_inline)) {
    const Group gr(plan.group[now / tiles]);
    const int n = now % tiles * 16 + r;
    if (slot < gr.count && n < I) {
      uint16_t hv[3];
      split3(g / (1.0f + expf(-g)) * u, hv);
      const int64_t at = (int64_t)(plan.pair[gr.first + slot] & 0xFFFFu) * I + n;
#pragma unroll
      for (int z = 0; z < 3; ++z) h[z * (int64_t)P * I + at] = hv[z];
    }
  };
  job.template run<TAIL>(
      smem + wave * S::kLds, H, JOIN ? wave : 0, JOIN ? 4 : 1, r < G ? r : 0, mine,
      [&](S& j) {
        if (ahead >= tasks) return false;
        const Group gr(plan.group[ahead / tiles]);
        const int n0 = ahead % tiles * 16, last = min(16, I - n0) - 1;
        const int64_t row = (int64_t)gr.expert * I + n0;
        const uint8_t* const c[2] = {gc + row * (H / 2), uc + row * (H / 2)};
        const uint8_t* const s[2] = {gs + row * mx4_scale_stride(H), us + row * mx4_scale_stride(H)};
        j.pieces = (gr.count + 1) / 2;
        j.init(H, c, s, [&](int, int i) { return min(i, last); }, x,
               [&](int m) { return (int)(plan.pair[gr.first + min(m, gr.count - 1)] >> 16); });
        ahead += step;
        return true;
      },
      [&](const f32x4_t(&acc)[2][1]) {
        if constexpr (JOIN) {
          auto& pt = part[(now - first) / step & 1];
          pt[wave][0][lane] = acc[0][0];
          pt[wave][1][lane] = acc[1][0];
          __syncthreads();
          // wave i finishes pair 4q + i of every quarter
          float g = 0.0f, u = 0.0f;
#pragma unroll
          for (int v = 0; v < 4; ++v) g += pt[v][0][lane][wave], u += pt[v][1][lane][wave];
          finish(g, u, 4 * q + wave);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) finish(acc[0][0][i], acc[1][0][i], 4 * q + i);
        }
        now += step;
      });
}

// y[t][n] = sum_j w[t][j] (down row n on h[t * k + j]).  A workgroup owns R tiles of 16 rows
// (blockIdx.x) and every gridDim.y-th lot of WAVES groups; its waves take one group after another, and
// each adds its products, times their weights, to token sums of its own in LDS, which are joined in wave
// order.  Row 4s + z of the matrix operand is plane z of pair s (LDS row 3s + z), so the planes' sums meet
// in one lane.  Where gridDim.y > 1, the workgroups of a tile leave their sums in `sums`
// [gridDim.y][T][H] at device scope, and the one that counts in last adds them up in order.
template <int R, int XP, int DEPTH, int WAVES, int TOKENS, bool SMALL, bool TAIL>
__global__ void __launch_bounds__(WAVES * 64) moe_down_kernel(int T, int k, int E, int H, int I,
    const uint16_t* __restrict__ h, const int32_t* __restrict__ ids, const float* __restrict__ weights,
    const uint8_t* __restrict__ dc, const uint8_t* __restrict__ ds, float* __restrict__ y, float* __restrict__ sums,
    uint32_t* __restrict__ counters) {
  constexpr int G = 2 * XP / 3, kCols = 16 * R;
  static_assert(G <= 4, "");
  using S = Skinny<1, R, XP, DEPTH>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WAVES * S::kLds];
  __shared__ typename Groups<SMALL ? 64 : kMaxPairs, G, true>::Storage plan;
  __shared__ float ysum[WAVES][TOKENS][kCols];
  __shared__ int done;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, r = lane & 15;
  const int P = T * k;
  for (int i = lane; i < T * kCols; i += 64) (&ysum[wave][0][0])[i] = 0.0f;
  const int groups = Groups<SMALL ? 64 : kMaxPairs, G, true>::find(P, E, k, ids, weights, plan, smem);
  const int n0 = blockIdx.x * kCols, last = min(kCols, H - n0) - 1;
  const int first = (int)blockIdx.y * WAVES + wave, step = WAVES * (int)gridDim.y;
  const int mine = groups > first ? (groups - 1 - first) / step + 1 : 0;
  S job;
  int ahead = first, now = first;
  job.template run<TAIL>(
      smem + wave * S::kLds, I, 0, 1, min(3 * (r >> 2) + min(r & 3, 2), 2 * XP - 1), mine,
      [&](S& j) {
        if (ahead >= groups) return false;
        const Group gr(plan.group[ahead]);
        const int64_t row = (int64_t)gr.expert * H + n0;
        const uint8_t* const c[1] = {dc + row * (I / 2)};
        const uint8_t* const s[1] = {ds + row * mx4_scale_stride(I)};
        j.pieces = (3 * gr.count + 1) / 2;
        j.init(I, c, s, [&](int t, int i) { return min(16 * t + i, last); }, h,
               [&](int m) { return m % 3 * P + (int)(plan.pair[gr.first + min(m / 3, gr.count - 1)] & 0xFFFFu); });
        ahead += step;
        return true;
      },
      [&](const f32x4_t(&acc)[1][R]) {
        const Group gr(plan.group[now]);
        const int at = gr.first + min(q, gr.count - 1), token = (int)(plan.pair[at] >> 16);
        const float w = plan.weight[at];
        // one quarter of the wave at a time: a token may hold the same expert twice
        for (int z = 0; z < gr.count; ++z) {
          if (q == z) {
#pragma unroll
            for (int t = 0; t < R; ++t) ysum[wave][token][16 * t + r] += w * ((acc[0][t][2] + acc[0][t][1]) + acc[0][t][0]);
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        now += step;
      });
  __syncthreads();
  const bool split = gridDim.y > 1;
  for (int i = threadIdx.x; i < T * kCols; i += WAVES * 64) {
    const int t = i / kCols, c = i % kCols;
    float s = ysum[0][t][c];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) s += ysum[v][t][c];
    if (c <= last) {
      if (split)
        __hip_atomic_store(sums + ((int64_t)blockIdx.y * T + t) * H + n0 + c, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      else
        y[(int64_t)t * H + n0 + c] = s;
    }
  }
  if (!split) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums are out
  __syncthreads();
  if (threadIdx.x == 0)
    done = __hip_atomic_fetch_add(counters + blockIdx.x, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.y - 1;
  __syncthreads();
  if (!done) return;
  for (int i = threadIdx.x; i < T * kCols; i += WAVES * 64) {
    const int t = i / kCols, c = i % kCols;
    if (c > last) continue;
    float s = 0.0f;
    for (int v0 = 0; v0 < (int)gridDim.y; v0 += 8) {
      float some[8];
#pragma unroll
      for (int v = 0; v < 8; ++v)
        some[v] = v0 + v < (int)gridDim.y ? __hip_atomic_load(sums + ((int64_t)(v0 + v) * T + t) * H + n0 + c,
                                                              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                          : 0.0f;
#pragma unroll
      for (int v = 0; v < 8; ++v) s += some[v];
    }
    y[(int64_t)t * H + n0 + c] = s;
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

// How the two kernels of a call are laid out.  xp: token pieces (two tokens each) of the first; split:
// workgroups that share a tile of the second; one: a single token, whose at most 16 experts fill the
// waves of one workgroup per tile.
struct MoePlan {
  int xp, tile_rows, tiles, split;
  bool one, small, join, few;
  int64_t hidden_bytes, sum_bytes, counter_bytes;
};

static MoePlan moe_plan(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  MoePlan m{};
  const int64_t P = T * k, most = P < E ? P : E;  // experts with pairs, at most
  m.small = P <= 64 && T <= 32;
  m.one = T == 1;
  m.few = T <= 32;
  m.xp = T <= 2 ? 1 : 2 * P <= 5 * most && P <= kFewPairs ? 2 : 4;
  // tasks for about one wave a SIMD, or fewer: four waves share one
  m.join = m.small && most * ((I + 15) / 16) <= 4 * (int64_t)device_cu_count();
  if (m.join && m.xp > 2) m.xp = 2;
  m.tile_rows = m.one ? 16 : 32;
  m.tiles = (int)((H + m.tile_rows - 1) / m.tile_rows);
  // the second kernel runs one workgroup a CU, each with a group for every wave
  int64_t split = m.one ? 1 : (int64_t)device_cu_count() / m.tiles;
  if (split > (most + 3) / 4) split = (most + 3) / 4;
  m.split = (int)(split < 1 ? 1 : split > 32 ? 32 : split);
  auto pad = [](int64_t b) { return (b + 255) / 256 * 256; };
  m.hidden_bytes = pad(3 * P * I * 2);
  m.sum_bytes = m.split > 1 ? pad((int64_t)m.split * T * H * 4) : 0;
  m.counter_bytes = m.split > 1 ? pad((int64_t)m.tiles * 4) : 0;
  return m;
}

size_t mx4_moe_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  const MoePlan m = moe_plan(T, k, E, H, I);
  return (size_t)(m.hidden_bytes + m.sum_bytes + m.counter_bytes);
}

namespace {

template <int XP, bool JOIN, bool SMALL>
void gate_up_as(const MoeArgs& a, const MoePlan& m, uint16_t* h, uint32_t* counters, hipStream_t stream) {
  // at most as many workgroups as run at a time, two a CU, and as tasks there can be
  const int64_t each = JOIN ? 1 : 4, tasks = ((int64_t)a.T * a.k * ((a.I + 15) / 16) + each - 1) / each;
  const int64_t slots = (XP == 2 ? 3 : 2) * (int64_t)device_cu_count();
  const auto kernel = a.H % (2 * kMxChunk) ? moe_gate_up_kernel<XP, JOIN, SMALL, true>
                                           : moe_gate_up_kernel<XP, JOIN, SMALL, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tasks < slots ? tasks : slots)), dim3(256), 0, stream, a.T, a.k, a.E, a.H, a.I,
                     a.x, a.ids, a.gate_codes, a.gate_scales, a.up_codes, a.up_scales, h, counters,
                     m.split > 1 ? m.tiles : 0);
}

template <int R, int XP, int DEPTH, int WAVES, int TOKENS, bool SMALL>
void down_as(const MoeArgs& a, const MoePlan& m, const uint16_t* h, float* sums, uint32_t* counters, hipStream_t stream) {
  const auto kernel = a.I % (2 * kMxChunk) ? moe_down_kernel<R, XP, DEPTH, WAVES, TOKENS, SMALL, true>
                                           : moe_down_kernel<R, XP, DEPTH, WAVES, TOKENS, SMALL, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)m.tiles, (unsigned)m.split), dim3(WAVES * 64), 0, stream, a.T, a.k, a.E, a.H,
                     a.I, h, a.ids, a.weights, a.down_codes, a.down_scales, a.y, sums, counters);
}

}  // namespace

hipError_t launch_mx4_moe(const MoeArgs& a, hipStream_t stream) {
  const MoePlan m = moe_plan(a.T, a.k, a.E, a.H, a.I);
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  uint16_t* h = reinterpret_cast<uint16_t*>(w);
  float* sums = reinterpret_cast<float*>(w + m.hidden_bytes);
  uint32_t* counters = reinterpret_cast<uint32_t*>(w + m.hidden_bytes + m.sum_bytes);
  if (m.join) {
    if (m.xp == 1) gate_up_as<1, true, true>(a, m, h, counters, stream);
    else gate_up_as<2, true, true>(a, m, h, counters, stream);
  } else if (m.xp == 1) gate_up_as<1, false, true>(a, m, h, counters, stream);
  else if (m.xp == 2) m.small ? gate_up_as<2, false, true>(a, m, h, counters, stream) : gate_up_as<2, false, false>(a, m, h, counters, stream);
  else m.small ? gate_up_as<4, false, true>(a, m, h, counters, stream) : gate_up_as<4, false, false>(a, m, h, counters, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (m.one) down_as<1, 2, 4, 8, 1, true>(a, m, h, sums, counters, stream);
  else if (m.small) down_as<2, 4, 2, 6, 32, true>(a, m, h, sums, counters, stream);
  else if (m.few) down_as<2, 4, 2, 6, 32, false>(a, m, h, sums, counters, stream);
  else down_as<2, 6, 2, 4, QL_MOE_MAX_TOKENS, false>(a, m, h, sums, counters, stream);
  return hipGetLastError();
}

}  // namespace ql
