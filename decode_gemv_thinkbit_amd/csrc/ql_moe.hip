// Mixture of experts for a few tokens: the router's choice, and the experts' products on MX4 weights.
#include <algorithm>
#include <cmath>

#include "ql_mx4.hpp"

namespace ql {
namespace {

// ---------------------------------------------------------------- router
// One wave per token: latency bounds (16 tokens of 64 experts, 8 taken: 3.4 us, 4096 of 128: 5.4; an
// empty launch takes 2), so everything stays in registers and crosses lanes in the vector unit.  Logits
// become unsigned keys of the same order (NaN and -inf become 0, which is never taken), lane l holds
// experts l, 64 + l, ...; each of the k rounds takes the wave's largest key and, among the lanes that
// hold it, the lowest expert.
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

// the sum over the lanes up to this one
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
  v += lanes_of<0x111, 0xF>(v);
  v += lanes_of<0x112, 0xF>(v);
  v += lanes_of<0x114, 0xF>(v);
  v += lanes_of<0x118, 0xF>(v);
  v += lanes_of<0x142, 0xA>(v);
  return v + lanes_of<0x143, 0xC>(v);
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
// to 64 pairs in registers, every wave for itself; more by counting, with three barriers, the last of which gives
// the scratch memory back.
constexpr int kMaxPairs = QL_MOE_MAX_TOKENS * QL_MOE_MAX_TOPK;
static_assert(kMaxPairs <= 1024 && QL_MOE_MAX_TOKENS <= 64 && QL_MOE_MAX_EXPERTS <= 1024, "records' bits");

template <int PAIRS, int G>  // PAIRS: 64, or the most there may be
struct Groups {
  static constexpr bool SMALL = PAIRS == 64;
  static constexpr int kSlots = SMALL ? 64 * G : PAIRS;
  struct Storage {
    uint32_t group[PAIRS];  // expert, pairs << 10, first slot << 16
    uint16_t pair[kSlots];  // pair, token << 10
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
  // All threads; returns the number of groups.
  static __device__ int find(int P, int E, int k, const int32_t* __restrict__ ids, Storage& st, uint8_t* scratch) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t below = (1ull << lane) - 1;
    if constexpr (SMALL) {
      const int raw = lane < P ? ids[lane] : -1, id = raw < E ? raw : -1;  // negative: none
      const uint64_t like = same(id, id >= 0, E);
      const int rank = __popcll(like & below), r0 = rank - rank % G;
      uint64_t from = like;  // the group's pairs and those behind it
      for (int i = 0; i < r0; ++i) from &= from - 1;
      const int lead = from ? __builtin_ctzll(from) : 0, size = min(G, (int)__popcll(from));
      const uint64_t firsts = __ballot(id >= 0 && rank == r0);
      const int group = __popcll(firsts & ((1ull << lead) - 1));
      if (id >= 0) {
        st.pair[group * G + rank % G] = (uint16_t)(lane | lane / k << 10);
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
          const int both = (int)wave_prefix((uint32_t)(n | ((n + G - 1) / G) << 16));
          if (e0 + lane < E) {
            const int before = both - (n | ((n + G - 1) / G) << 16);
            sc.start[e0 + lane] = (uint32_t)(slots + (before & 0xFFFF)) | (uint32_t)(groups + (before >> 16)) << 16;
          }
          const int all = __builtin_amdgcn_readlane(both, 63);
          slots += all & 0xFFFF, groups += all >> 16;
        }
        if (lane == 0) st.groups = groups;
      }
      __syncthreads();
      for (int p = threadIdx.x; p < P; p += blockDim.x) {
        const int e = sc.id[p], rank = sc.rank[p];
        if (e == 65535) continue;
        const int slot = (int)(sc.start[e] & 0xFFFF) + rank, group = (int)(sc.start[e] >> 16) + rank / G;
        st.pair[slot] = (uint16_t)(p | p / k << 10);
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

// A wave's first task: the first waves of all workgroups, then the second ones, ..., so that a last, partly
// filled round loads every CU alike.  Workgroups go round the XCDs: those of one XCD take neighbouring
// tasks, whose rows meet in a cache line where their bytes are no multiple of 128 (gate and up of 128 x 736 x
// 2080, 6 for 24 tokens: 37.5 us without, 34.0 with; 43.9 with neighbours in one workgroup).
__device__ __forceinline__ int first_task(int wave) {
  const int grid = (int)gridDim.x, block = (int)blockIdx.x;
  return wave * grid + (grid % 8 ? block : block % 8 * (grid / 8) + block / 8);
}

// The three bf16 planes of an fp32 value: hi + mid + lo == v from 2^-110 up (the second product then runs on
// exact bf16 operands), below to half of 2^-133, the last plane's least step.  Where hi would round past the
// largest bf16 (0x7F7F8000 and above) it is cut off instead, and the 16 bits left still fit the other two; of
// a value that is not finite only the first is kept.
__device__ __forceinline__ void split3(float v, uint16_t (&h)[3]) {
  const uint32_t b = __float_as_uint(v);
  h[0] = (b & 0x7FFFFFFFu) - 0x7F7F8000u < 0x8000u ? (uint16_t)(b >> 16) : f32_to_bf16_bits(v);
  const float r = v - bf16_bits_to_f32(h[0]);
  const bool fine = (h[0] & 0x7F80u) != 0x7F80u;
  h[1] = fine ? f32_to_bf16_bits(r) : 0;
  h[2] = fine ? f32_to_bf16_bits(r - bf16_bits_to_f32(h[1])) : 0;
}

// silu(g) * u, silu(g) = g / (1 + exp(-g)).  Below -88, where exp(-g) overflows although the product need not
// vanish, 1 + exp(-g) is exp(-g) to fp32, and exp(g) is taken in two halves, which stay in range.
__device__ __forceinline__ float swiglu(float g, float u) {
  if (g < -88.0f) {
    const float t = expf(0.5f * g);
    return (g * t) * (t * u);
  }
  return g / (1.0f + expf(-g)) * u;
}

// h[p][i] = silu(g) * u with g, u the gate's and the up projection's row i on pair p's token.  A task is 16
// rows of both for one group.  JOIN (few tasks): workgroups take tasks in turn, the inputs' pairs of
// chunks dealt to the four waves and their sums joined in wave order; else every wave takes tasks of its
// own.  Either way the next task's loads are under way while one ends.  The stream of the experts' rows
// bounds: traced, with weights from HBM, 57 experts of 1536 x 4096 (376 MB) take 74 us, 5.1 TB/s; 87 of 768 x 2048
// (146 MB) 30 us, 4.9; 88 of 736 x 2080, whose rows are no whole cache lines, 37 us, 3.9.
template <int XP, int WAVES, bool JOIN, bool SMALL, bool TAIL>
__global__ void __launch_bounds__(WAVES * 64) moe_gate_up_kernel(int T, int k, int E, int H, int I,
    const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint8_t* __restrict__ gc,
    const uint8_t* __restrict__ gs, const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us,
    uint16_t* __restrict__ h) {
  constexpr int G = 2 * XP, kPairs = SMALL ? 64 : kMaxPairs;
  using S = Skinny<2, 1, XP>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WAVES * S::kLds];
  __shared__ typename Groups<kPairs, G>::Storage plan;
  __shared__ f32x4_t part[JOIN ? 2 : 1][JOIN ? 4 : 1][2][64];
  static_assert(!JOIN || WAVES == 4, "wave i finishes row i of every quarter");
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int P = T * k, tiles = (I + 15) / 16;
  const int tasks = Groups<kPairs, G>::find(P, E, k, ids, plan, smem) * tiles;
  const int first = JOIN ? (int)blockIdx.x : first_task(wave), step = (JOIN ? 1 : WAVES) * (int)gridDim.x;
  const int mine = tasks > first ? (tasks - 1 - first) / step + 1 : 0;
  S job;
  int ahead = first, now = first;
  auto finish = [&](float g, float u, int slot) __attribute__((always_inline)) {
    const Group gr(plan.group[now / tiles]);
    const int n = now % tiles * 16 + r;
    if (slot < gr.count && n < I) {
      uint16_t hv[3];
      split3(swiglu(g, u), hv);
      const int64_t at = (int64_t)(plan.pair[gr.first + slot] & 1023) * I + n;
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
               [&](int m) { return plan.pair[gr.first + min(m, gr.count - 1)] >> 10; });
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

// The down projection's operand: row 4s + z of the matrix instruction is plane z of a group's pair s (LDS row
// 3s + z), so the planes' sums meet in one lane, smallest first.
template <int XP>
__device__ __forceinline__ int plane_row(int r) { return min(3 * (r >> 2) + min(r & 3, 2), 2 * XP - 1); }
__device__ __forceinline__ float planes(const f32x4_t& v) { return (v[2] + v[1]) + v[0]; }

// products[s][p][n] = part s of down row n on h[p].  A task is R tiles of 16 rows for one group; every wave
// takes tasks of its own, or `split` (which divides WAVES) waves each a part of a task's pairs of chunks.
// What a CU fetches bounds: a row of W is 17/32 bytes an input, three planes of up to four pairs up to 24
// (traced, from HBM, 4096 x 1536 for 57 experts, 190 MB, 44 us; 2048 x 768 for 87 19 us; 4 tiles a task halve the
// planes' share).
template <int R, int XP, int WAVES, int PAIRS, bool TAIL>
__global__ void __launch_bounds__(WAVES * 64) moe_down_kernel(int T, int k, int E, int H, int I, int split,
    const uint16_t* __restrict__ h, const int32_t* __restrict__ ids, const uint8_t* __restrict__ dc,
    const uint8_t* __restrict__ ds, float* __restrict__ products) {
  constexpr int G = 2 * XP / 3;
  static_assert(G <= 4, "");
  using S = Skinny<1, R, XP>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WAVES * S::kLds];
  __shared__ typename Groups<PAIRS, G>::Storage plan;
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int P = T * k, tiles = (H + 16 * R - 1) / (16 * R);
  const int tasks = Groups<PAIRS, G>::find(P, E, k, ids, plan, smem) * tiles;
  const int first = first_task(wave / split), step = WAVES / split * (int)gridDim.x;
  const int mine = tasks > first ? (tasks - 1 - first) / step + 1 : 0;
  products += (int64_t)(wave % split) * P * H;
  S job;
  int ahead = first, now = first;
  job.template run<TAIL>(
      smem + wave * S::kLds, I, wave % split, split, plane_row<XP>(r), mine,
      [&](S& j) {
        if (ahead >= tasks) return false;
        const Group gr(plan.group[ahead / tiles]);
        const int n0 = ahead % tiles * (16 * R), last = min(16 * R, H - n0) - 1;
        const int64_t row = (int64_t)gr.expert * H + n0;
        const uint8_t* const c[1] = {dc + row * (I / 2)};
        const uint8_t* const s[1] = {ds + row * mx4_scale_stride(I)};
        j.pieces = (3 * gr.count + 1) / 2;
        j.init(I, c, s, [&](int t, int i) { return min(16 * t + i, last); }, h,
               [&](int m) { return m % 3 * P + (plan.pair[gr.first + min(m / 3, gr.count - 1)] & 1023); });
        ahead += step;
        return true;
      },
      [&](const f32x4_t(&acc)[1][R]) {
        const Group gr(plan.group[now / tiles]);
        const int n = now % tiles * (16 * R) + r;
        if (q < gr.count) {
          float* out = products + (int64_t)(plan.pair[gr.first + q] & 1023) * H + n;
#pragma unroll
          for (int t = 0; t < R; ++t)
            if (n + 16 * t < H) out[16 * t] = planes(acc[0][t]);
        }
        now += step;
      });
}

// y[t][n] = sum_j weights[t][j] sum_s products[s][t * k + j][n], over the pairs with an expert, in order: four
// outputs a thread.
__global__ void __launch_bounds__(256) moe_join_kernel(int T, int k, int E, int H, int split,
                                                       const int32_t* __restrict__ ids, const float* __restrict__ weights,
                                                       const float* __restrict__ products, float* __restrict__ y) {
  const int t = blockIdx.y, n = 4 * (int)(blockIdx.x * 256 + threadIdx.x);
  if (n >= H) return;
  f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = 0; j0 < k; j0 += 8) {
    f32x4_t v[8];
    const float* from = products + (int64_t)t * k * H + n;
#pragma unroll
    for (int j = 0; j < 8; ++j)  // pairs without an expert hold nothing: read, for one round of loads, and left out
      v[j] = *reinterpret_cast<const f32x4_t*>(from + (int64_t)min(j0 + j, k - 1) * H);
    for (int s = 1; s < split; ++s) {
      from += (int64_t)T * k * H;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += *reinterpret_cast<const f32x4_t*>(from + (int64_t)min(j0 + j, k - 1) * H);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = t * k + min(j0 + j, k - 1), id = ids[p];
      const float w = weights[p];
      const bool is = j0 + j < k && id >= 0 && id < E;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += is ? w * v[j][i] : 0.0f;
    }
  }
  *reinterpret_cast<f32x4_t*>(y + (int64_t)t * H + n) = sum;
}

// One token: its experts (at most 16) fill the waves of one workgroup per 16 rows, `split` of them to an
// expert, dealt its pairs of chunks in turn; their sums are joined in wave order.  No second pass.
template <bool TAIL>
__global__ void __launch_bounds__(1024) moe_down_one_kernel(int k, int E, int H, int I, int split,
    const uint16_t* __restrict__ h, const int32_t* __restrict__ ids, const float* __restrict__ weights,
    const uint8_t* __restrict__ dc, const uint8_t* __restrict__ ds, float* __restrict__ y) {
  using S = Skinny<1, 1, 2>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[16 * S::kLds];
  __shared__ float part[16][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15;
  const int n0 = blockIdx.x * 16, pair = wave / split;
  const int id = pair < k ? ids[pair] : -1;
  const bool is = id >= 0 && id < E;
  float sum = 0.0f;
  bool once = is;
  S job;
  job.template run<TAIL>(
      smem + wave * S::kLds, I, wave % split, split, plane_row<2>(r), is ? 1 : 0,
      [&](S& j) {
        if (!once) return false;
        once = false;
        const int64_t row = (int64_t)id * H + n0;
        const uint8_t* const c[1] = {dc + row * (I / 2)};
        const uint8_t* const s[1] = {ds + row * mx4_scale_stride(I)};
        j.init(I, c, s, [](int, int i) { return i; }, h, [&](int m) { return min(m, 2) * k + pair; });
        return true;
      },
      [&](const f32x4_t(&acc)[1][1]) { sum = planes(acc[0][0]); });
  if (lane < 16) part[wave][r] = sum;
  __syncthreads();
  if (threadIdx.x < 16) {
    float all = 0.0f;
    for (int j = 0; j < k; ++j) {
      float v = part[j * split][r];
      for (int u = 1; u < split; ++u) v += part[j * split + u][r];
      if (ids[j] >= 0 && ids[j] < E) all += weights[j] * v;
    }
    y[n0 + r] = all;
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

// How a call's kernels are laid out.
//   one: a single token, whose experts fill the waves of a workgroup (8 of 64 experts of 1024 x 2048: 4.7 us
//     against the 8.8 of products and their join).
//   xp: token pieces (two tokens each) of the first kernel: two tokens need one; up to 16 else, as an expert
//     with more pairs than a group holds is read again (128 experts of 1536 x 4096, 8 for 64 tokens: 176 us,
//     with groups of 8 180, of 4 211; few pairs an expert cost nothing, as pieces without a token are not
//     loaded).
//   join: too few tasks for a wave on every SIMD: four waves share one (8 experts of 1024 x 2048: 6.8 us
//     against 8.2; of 1536 x 4096 12.2 against 17.4; 15 of 1024 x 2048, about the bound, 9.1 both); its groups
//     hold four pairs, so not where experts have more (2 of 4096 x 2048 for 64 tokens: 23.5 us, 12.0 without).
//   wide: tasks of 64 rows in the second kernel where that leaves each wave three or more (those 128 experts:
//     104 us against 118; 8 of 14336 x 4096, 2 for 64 tokens, on the other side, 207 against 178).
//   split: waves that share a task of the second, where tasks are few and rows long (3 experts of 14336 x 4096:
//     25 us against 49).
//   gate_waves, down_waves: of a workgroup, one to a CU.  Fewer keep the lines that two rows share in the L2 and
//     contend less; as many as LDS holds (11 and 12) are taken up to 64 pairs (10 tokens, 6 of 128 experts of 736 x
//     2080: 40.5 us, with 9 and 10 42.4), and above where the tasks that T tokens with k of E experts each make on
//     average need one round for two or two for three (9, 8 of 60 of 1024 x 2048, 2780 tasks: 41.1 against 43.4;
//     24, 8 of 128 of 768 x 2048: 60.6 against 62.9; 20, 4 of 32 of 1408 x 2048: 41.8 against 45.4; with as many
//     rounds 16, 8 of 60 of 1024 x 2048: 51.2 against 50.2, 32, 8 of 64 of 1536 x 4096: 155.5 against 151.1; five
//     for six, 64, 8 of 128 of 1536 x 4096: 289 against 284).  In the second kernel only a single round is worth it
//     (those 9 tokens: 1.1 us; 24, 6 of 128 of 736 x 2080, two rounds for three: 0.6 us the other way).
constexpr int kGateWaves = 11, kGateFewer = 9, kDownWaves = 12, kDownFewer = 10, kWideWaves = 8;

MoePlan moe_plan(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  MoePlan m{};
  const int64_t cus = device_cu_count();
  const int64_t P = T * k, most = P < E ? P : E;  // experts with pairs, at most
  m.small = P <= 64;
  m.one = T == 1;
  m.xp = T <= 2 ? 1 : 8;
  m.join = m.small && P <= 4 * most && most * ((I + 15) / 16) <= 4 * cus;
  if (m.join && m.xp > 1) m.xp = 2;
  const int64_t groups = most > P / 4 ? most : P / 4;  // of the second kernel, about
  m.wide = !m.small && groups * ((H + 63) / 64) >= 3 * kWideWaves * cus;
  m.split = 1;
  if (m.small)
    for (int split : {2, 3, 4, 6, 12})
      if (I >= 1024 * split && most * ((H + 31) / 32) * split <= kDownWaves * cus) m.split = split;
  m.gate_waves = m.join ? 4 : m.xp == 1 ? 16 : kGateWaves;
  m.down_waves = m.one ? (int)k * (16 / (int)k) : m.wide ? kWideWaves : kDownWaves;
  if (!m.small) {
    const double mean = (double)E * (1.0 - std::pow(1.0 - (double)k / (double)E, (double)T));  // experts with pairs
    auto tasks = [&](int64_t group, int64_t tiles) { return (int64_t)(std::max(mean, (double)(P / group)) * tiles); };
    auto rounds = [&](int64_t n, int waves) { return (n + waves * cus - 1) / (waves * cus); };
    const int64_t gate = tasks(16, (I + 15) / 16), down = tasks(4, (H + 31) / 32);
    if (rounds(gate, kGateWaves) > 2 || rounds(gate, kGateFewer) == rounds(gate, kGateWaves)) m.gate_waves = kGateFewer;
    if (!m.wide && (down > kDownWaves * cus || down <= kDownFewer * cus)) m.down_waves = kDownFewer;
  }
  auto pad = [](int64_t b) { return (b + 255) / 256 * 256; };
  m.hidden_bytes = pad(3 * P * I * 2);
  m.product_bytes = m.one ? 0 : pad(m.split * P * H * 4);
  return m;
}

size_t mx4_moe_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  const MoePlan m = moe_plan(T, k, E, H, I);
  return (size_t)(m.hidden_bytes + m.product_bytes);
}

namespace {

// As many workgroups as run at a time, or as tasks there can be
template <int XP, int WAVES, bool JOIN, bool SMALL>
void gate_up_as(const MoeArgs& a, uint16_t* h, hipStream_t stream) {
  const int64_t tasks = (int64_t)a.T * a.k * ((a.I + 15) / 16);
  const int64_t slots = (JOIN ? XP == 1 ? 4 : 3 : 1) * (int64_t)device_cu_count();
  const auto kernel = a.H % (2 * kMxChunk) ? moe_gate_up_kernel<XP, WAVES, JOIN, SMALL, true>
                                           : moe_gate_up_kernel<XP, WAVES, JOIN, SMALL, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tasks < slots ? tasks : slots)), dim3(WAVES * 64), 0, stream, a.T, a.k, a.E,
                     a.H, a.I, a.x, a.ids, a.gate_codes, a.gate_scales, a.up_codes, a.up_scales, h);
}

template <int R, int XP, int WAVES, int PAIRS>
void down_as(const MoeArgs& a, int split, const uint16_t* h, float* products, hipStream_t stream) {
  const int64_t tasks = (int64_t)a.T * a.k * ((a.H + 16 * R - 1) / (16 * R)), slots = device_cu_count();
  const auto kernel = a.I % (2 * kMxChunk) ? moe_down_kernel<R, XP, WAVES, PAIRS, true>
                                           : moe_down_kernel<R, XP, WAVES, PAIRS, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tasks < slots ? tasks : slots)), dim3(WAVES * 64), 0, stream, a.T, a.k, a.E,
                     a.H, a.I, split, h, a.ids, a.down_codes, a.down_scales, products);
}

}  // namespace

hipError_t launch_mx4_moe(const MoeArgs& a, hipStream_t stream) {
  const MoePlan m = moe_plan(a.T, a.k, a.E, a.H, a.I);
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  uint16_t* h = reinterpret_cast<uint16_t*>(w);
  float* products = reinterpret_cast<float*>(w + m.hidden_bytes);
  if (m.join && m.xp == 1) gate_up_as<1, 4, true, true>(a, h, stream);
  else if (m.join) gate_up_as<2, 4, true, true>(a, h, stream);
  else if (m.xp == 1) gate_up_as<1, 16, false, true>(a, h, stream);
  else if (m.small) gate_up_as<8, kGateWaves, false, true>(a, h, stream);
  else if (m.gate_waves == kGateWaves) gate_up_as<8, kGateWaves, false, false>(a, h, stream);
  else gate_up_as<8, kGateFewer, false, false>(a, h, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (m.one) {
    const auto kernel = a.I % (2 * kMxChunk) ? moe_down_one_kernel<true> : moe_down_one_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(a.H / 16)), dim3((unsigned)(m.down_waves * 64)), 0, stream, a.k, a.E, a.H,
                       a.I, m.down_waves / a.k, h, a.ids, a.weights, a.down_codes, a.down_scales, a.y);
    return hipGetLastError();
  }
  if (m.small) down_as<2, 6, kDownWaves, 64>(a, m.split, h, products, stream);
  else if (m.wide) down_as<4, 6, kWideWaves, kMaxPairs>(a, m.split, h, products, stream);
  else if (m.down_waves == kDownWaves) down_as<2, 6, kDownWaves, kMaxPairs>(a, m.split, h, products, stream);
  else down_as<2, 6, kDownFewer, kMaxPairs>(a, m.split, h, products, stream);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((a.H / 4 + 255) / 256), (unsigned)a.T), dim3(256), 0, stream, a.T,
                     a.k, a.E, a.H, m.split, a.ids, a.weights, products, a.y);
  return hipGetLastError();
}

}  // namespace ql
