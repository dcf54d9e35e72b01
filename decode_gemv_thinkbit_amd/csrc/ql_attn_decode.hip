// Attention of one new token per sequence over the paged cache.
//
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale * q . k_j,  m = max_j s_j,
//
// in one pass over the keys: m, the sum and o are kept for the keys seen so far, and o and the sum are scaled
// down when m grows.  The G = Hq / Hkv heads that share a kv head are the columns of the matrix instructions,
// so the cache is read once (once per 16 heads, if G is above 16).
//
// v_mfma_f32_16x16x32_bf16: lane (q, r) = (lane / 16, lane % 16) holds eight inputs of row (or column) r, and
// rows 4q .. 4q + 3 of column r of the result.  A wave takes 32 keys a step:
//  - scores of keys x heads (K is the first operand): tile t's row r is key 8 (r / 4) + r % 4 + 4 t, so lane
//    (q, r) gets head r's scores of keys 8q .. 8q + 7: what the second product wants of it;
//  - output of dims x heads (V is the first operand): instruction i's row r is dim (D / 16) r + i, so lane
//    (q, r) reads of keys 8q .. 8q + 7 the D / 16 dims from (D / 16) r on, whole rows by 16 lanes, and a byte
//    permute of two keys' dwords makes each operand.  Neither K nor V goes through LDS.
//
// Reading the cache bounds.  131072 keys of 8 heads of 128 in bf16 (537 MB) take 80.7 us, 6.6 of the 7.0 TB/s that a
// pure read reaches, and 87.5 with the join; 64 sequences of 0 .. 8192 keys (253 MB) 48 and 55: a CU fetches at most
// 35 KB a microsecond, 1.4 times its share, so CUs that got more than others end late.  What that led to:
//  - keys and values are read past the caches (nontemporal): 105.7 -> 94.0 us for the 131072 keys;
//  - one step's loads at a time and four workgroups a CU, not two steps' and two: 62 -> 55 us for the 64 sequences,
//    no difference for long ones (registers: 128, a wave more or less of them decides);
//  - chunks of equal length, of four waves: equal shares of all sequences' keys, cut anywhere, balance better but wait
//    at every sequence's end (55.3 us; 33 sequences of heads of 64: 13.7 us against 9.6); full chunks before the
//    sequences' rests made no difference, nor did shorter or longer chunks (53.5 .. 67 us).
#include <algorithm>

#include "ql_attn.hpp"

namespace ql {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;                    // keys of a wave's step
constexpr int kChunkStep = kWaves * kStep;   // a chunk's keys are a multiple: one step of each wave
// Where no sequence can have more keys, each is one chunk and nothing is joined.  Up to 500 keys of one sequence, 32 over 8
// heads: 8.0 us so and 8.2 in chunks of 128 keys; of 64 sequences 12.1 and 13.9; with 1000 keys 16.6 and 8.2.
constexpr int kWhole = 512;
constexpr int kTarget = 1024;                // chunks of a call, about: four workgroups for each CU
constexpr int kRows = 16;                    // heads a workgroup takes at most

// Work is cut on the device, where the lengths are: chunks of equal length C over all sequences, C the least
// (a multiple of kChunkStep) for which the grid, kTarget + one for each sequence and head, holds them all.
// Every wave finds its place by itself, 256 sequences at a time.
struct Place {
  int b, len, chunk, chunks, first, size;  // first: the number of b's first chunk; size: keys of a chunk
};
__device__ __forceinline__ int clamp_len(int len, int keys) { return len < 0 ? 0 : len > keys ? keys : len; }

// The sequence that has chunk number `want` (b < 0: none)
__device__ __forceinline__ Place find_place(const int32_t* __restrict__ lens, int B, int keys, int heads, int want) {
  const int lane = threadIdx.x & 63;
  int len[4];  // of sequences b0 + 64 i + lane; -1: none
  auto read = [&](int b0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + 64 * i + lane;
      len[i] = b < B ? lens[b] : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) len[i] = b0 + 64 * i + lane < B ? clamp_len(len[i], keys) : -1;
  };
  auto steps = [](int n) { return n < 0 ? 0u : max(1u, ((uint32_t)n + kChunkStep - 1) / kChunkStep); };
  uint32_t total = 0;
  for (int b0 = (B - 1) & ~255; b0 >= 0; b0 -= 256) {  // ends with the first ones read
    read(b0);
    total += last_lane(scan_lanes(steps(len[0]) + steps(len[1]) + steps(len[2]) + steps(len[3])));
  }
  // (2^23 steps hold the longest sequence)
  const uint32_t c = (uint32_t)min(((uint64_t)total * (uint32_t)heads + kTarget - 1) / kTarget, (uint64_t)1 << 23);
  uint32_t before = 0;
  for (int b0 = 0; b0 < B; b0 += 256) {
    if (b0) read(b0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (b0 + 64 * i >= B) break;
      const uint32_t n = (steps(len[i]) + c - 1) / c, upto = before + scan_lanes(n);
      const uint64_t here = __ballot((uint32_t)want < upto);
      if (here) {
        const int l = __builtin_ctzll(here);
        Place p;
        p.b = b0 + 64 * i + l;
        p.len = __builtin_amdgcn_readlane(len[i], l);
        p.chunks = __builtin_amdgcn_readlane((int)n, l);
        p.first = __builtin_amdgcn_readlane((int)upto, l) - p.chunks;
        p.chunk = want - p.first;
        p.size = (int)c * kChunkStep;
        return p;
      }
      before = last_lane(upto);
    }
  }
  return Place{-1, 0, 0, 0, 0, 0};
}

struct Split {  // the grid of a call
  int G, tiles, rows, heads;  // heads: kv heads x tiles of 16 of their q heads; rows: of a tile
  int64_t units;
};
Split split_of(int64_t B, int64_t Hq, int64_t Hkv) {
  Split s;
  s.G = (int)(Hq / Hkv), s.tiles = (s.G + kRows - 1) / kRows, s.rows = std::min(s.G, kRows);
  s.heads = (int)Hkv * s.tiles;
  s.units = kTarget + B * s.heads;
  return s;
}
bool may_split(int64_t keys) { return keys > kWhole; }

// The workspace: [unit][row][D] sums of exp2(s - m) v, [unit][row][2] m and sum; then, for the joining kernel, the
// keys of a chunk and every sequence's first chunk (where it has more than one).
__host__ __device__ inline int64_t stats_at(const Split& sp, int D) { return sp.units * sp.rows * D; }
__host__ __device__ inline int64_t plan_at(const Split& sp, int D) { return sp.units * sp.rows * (D + 2); }

template <int D, bool F8, bool SPLIT>
__global__ void __launch_bounds__(64 * kWaves, 4) attn_decode_kernel(AttnArgs a, Split sp) {
  constexpr int ES = F8 ? 1 : 2;
  constexpr int KL = D * ES / 64;   // 16-byte loads of a key row by four lanes
  constexpr int NB = D / 16;        // dims of a lane in the second product, and its instructions
  constexpr int VD = NB * ES / 4;   // dwords of them as stored
  constexpr int NW = NB / 2;        // and as bf16
  __shared__ __attribute__((aligned(16))) float part[kWaves][kRows][D + 4];
  __shared__ float stats[kWaves][kRows][2];
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = blockIdx.x, hk = unit % sp.heads, head = hk / sp.tiles, tile = hk % sp.tiles;
  Place at;
  if constexpr (SPLIT) {
    at = find_place(a.lens, a.B, a.keys, sp.heads, unit / sp.heads);
    if (at.b < 0) return;
  } else {
    const int b = unit / sp.heads, len = clamp_len(a.lens[b], a.keys);
    at = Place{b, len, 0, 1, b, kWhole};
  }
  const int begin = at.chunk * at.size, end = min(at.len, begin + at.size);
  const int steps = (end - begin + kStep - 1) / kStep, mine = steps > wave ? (steps - wave + kWaves - 1) / kWaves : 0;
  const int rows = min(sp.rows, sp.G - tile * kRows);

  // q: column r, dims as K's bytes lie: 16 of a 64-byte piece to each lane
  uint32_t qw[D / 32][4];
  {
    const uint16_t* p = a.q + ((int64_t)at.b * a.Hq + (int64_t)head * sp.G + tile * kRows + min(r, rows - 1)) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int d = F8 ? 64 * (i / 2) + 16 * q + 8 * (i % 2) : 32 * i + 8 * q;
      const u32x4_t v = *(gu32x4p)(p + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) qw[i][j] = r < rows ? v[j] : 0u;
    }
  }
  const float c = a.score_scale * (a.kv.k_scale ? a.kv.k_scale[head] : 1.0f);
  const float room = room_of(at.len, 0.0f);

  const int32_t* __restrict__ row = a.table + at.b * a.table_stride;
  const int shift = a.kv.page_shift;
  const uint32_t row_bytes = D * ES;
  // Pages of a step's two halves of 16 keys (a page holds 16 or more).  The second half may begin behind the last
  // key; then the first's page stands for it.  Entries that are no page count as masked keys, page 0 is read.
  auto pages_of = [&](int s, int (&e)[2]) {
    const int k0 = begin + s * kStep, k1 = k0 + 16 < end ? k0 + 16 : k0;
    e[0] = row[k0 >> shift], e[1] = row[k1 >> shift];
  };
  u32x4_t kr[2][KL];
  uint32_t vr[8][VD];
  auto load = [&](int s, const int (&e)[2]) {
    const int k0 = begin + s * kStep;
    const uint8_t *kp[2], *vp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t page = (uint32_t)e[i] < (uint32_t)a.kv.pages ? e[i] : 0;
      const int64_t off = ((page * a.kv.heads + head) << shift) * row_bytes;
      kp[i] = a.kv.k + off, vp[i] = a.kv.v + off;
    }
    const uint32_t in = (1u << shift) - 1;
    const int key = k0 + 8 * (r >> 2) + (r & 3);  // tile 0's; tile 1's is 4 on
    const uint8_t* p = (r >> 3 ? kp[1] : kp[0]) + (key & in) * row_bytes + 16 * q;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < KL; ++i) kr[t][i] = load_once((gu32x4p)(p + t * 4 * row_bytes + i * 64));
    const uint8_t* v = (q >> 1 ? vp[1] : vp[0]) + ((k0 + 8 * q) & in) * row_bytes + r * (NB * ES);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (VD == 4) {
        const u32x4_t w = load_once((gu32x4p)(v + i * row_bytes));
#pragma unroll
        for (int j = 0; j < 4; ++j) vr[i][j] = w[j];
      } else if constexpr (VD == 2) {
        typedef const __attribute__((address_space(1))) u32x2_t* gu32x2p;
        const u32x2_t w = load_once((gu32x2p)(v + i * row_bytes));
        vr[i][0] = w[0], vr[i][1] = w[1];
      } else {
        typedef const __attribute__((address_space(1))) uint32_t* gu32p;
        vr[i][0] = load_once((gu32p)(v + i * row_bytes));
      }
    }
  };

  float m = kNegInf, sum = 0.0f;
  at_f32x4 o[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) o[i] = at_f32x4{0, 0, 0, 0};

  int e[2] = {0, 0}, ahead[2] = {0, 0};
  if (mine > 0) pages_of(wave, ahead);
  for (int n = 0; n < mine; ++n) {
    const int s = wave + kWaves * n;
    e[0] = ahead[0], e[1] = ahead[1];
    load(s, e);
    if (n + 1 < mine) pages_of(s + kWaves, ahead);
    // scores
    at_f32x4 sc[2] = {at_f32x4{0, 0, 0, 0}, at_f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const at_bf16x8 qv = __builtin_bit_cast(at_bf16x8, (u32x4_t{qw[i][0], qw[i][1], qw[i][2], qw[i][3]}));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4_t kv;
        if constexpr (F8) {
          const u32x2_t lo = bf16_of_e4m3(kr[t][i / 2][2 * (i % 2)]), hi = bf16_of_e4m3(kr[t][i / 2][2 * (i % 2) + 1]);
          kv = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
        } else {
          kv = kr[t][i];
        }
        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(at_bf16x8, kv), qv, sc[t], 0, 0, 0);
      }
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = sc[i / 4][i % 4] * c;
    uint32_t vw[8][NW];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < VD; ++j) {
          const u32x2_t w = bf16_of_e4m3(vr[i][j]);
          vw[i][2 * j] = w[0], vw[i][2 * j + 1] = w[1];
        }
      } else {
#pragma unroll
        for (int j = 0; j < NW; ++j) vw[i][j] = vr[i][j];
      }
    }
    // Keys behind the end or of no page: out of the maximum and the sum, their values (whatever the memory
    // holds, NaN too) taken as 0
    const int k0 = begin + s * kStep;
    const bool ok0 = (uint32_t)e[0] < (uint32_t)a.kv.pages, ok1 = (uint32_t)e[1] < (uint32_t)a.kv.pages;
    if (!(k0 + kStep <= end && ok0 && ok1)) {
      const bool ok = q >> 1 ? ok1 : ok0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool sees = ok && k0 + 8 * q + i < end;
        p[i] = sees ? p[i] : kNegInf;
#pragma unroll
        for (int j = 0; j < NW; ++j) vw[i][j] = sees ? vw[i][j] : 0u;
      }
    }
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, p[i]);
    top = max_xor32(max_xor16(top));
    const float m_new = fmaxf(m, top);
    const float alpha = part_weight(m, m_new);
    m = m_new;
    const float base = m == kNegInf ? 0.0f : m + room;
    sum *= alpha;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] *= alpha;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp2_fast(p[i] - base);
      sum += p[i];
    }
    // exp2 rounded to bf16, half a step of 2^-8 each; the sum is of the unrounded ones
    const u32x4_t pw{pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])};
    const at_bf16x8 pv = __builtin_bit_cast(at_bf16x8, pw);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      u32x4_t f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        f[k] = __builtin_amdgcn_perm(vw[2 * k + 1][i / 2], vw[2 * k][i / 2], i % 2 ? 0x07060302u : 0x05040100u);
      o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(at_bf16x8, f), pv, o[i], 0, 0, 0);
    }
  }

  // the waves' sums, joined in their order
  sum = sum_xor32(sum_xor16(sum));
  if (r < rows) {
    if (q == 0) stats[wave][r][0] = m, stats[wave][r][1] = sum;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < NB; i += 4)
        *(at_f32x4*)&part[wave][r][NB * (4 * q + j) + i] = at_f32x4{o[i][j], o[i + 1][j], o[i + 2][j], o[i + 3][j]};
  }
  __syncthreads();
  const bool whole = at.chunks == 1;
  if (SPLIT && threadIdx.x == 0 && hk == 0 && at.chunk == 0) {
    int32_t* plan = (int32_t*)(a.ws + plan_at(sp, D));
    if (at.first == 0) plan[0] = at.size;
    plan[1 + at.b] = at.first;
  }
  const float vs = whole && a.kv.v_scale ? a.kv.v_scale[head] : 1.0f;
  for (int idx = threadIdx.x; idx < rows * (D / 2); idx += 64 * kWaves) {
    const int g = idx / (D / 2), d = idx % (D / 2) * 2;
    float most = stats[0][g][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) most = fmaxf(most, stats[w][g][0]);
    float total = 0.0f, y0 = 0.0f, y1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = part_weight(stats[w][g][0], most);
      total += f * stats[w][g][1];
      y0 += f * part[w][g][d];
      y1 += f * part[w][g][d + 1];
    }
    if (whole) {
      const float inv = total == 0.0f ? 0.0f : vs / total;
      uint16_t* out = a.out + ((int64_t)at.b * a.Hq + (int64_t)head * sp.G + tile * kRows + g) * D + d;
      *(uint32_t*)out = pack_bf16(y0 * inv, y1 * inv);
    } else {
      float* out = a.ws + ((int64_t)unit * sp.rows + g) * D + d;
      *(float2*)out = make_float2(y0, y1);
      if (d == 0) *(float2*)(a.ws + stats_at(sp, D) + ((int64_t)unit * sp.rows + g) * 2) = make_float2(most, total);
    }
  }
}

// One workgroup for each sequence, head and slice of its dims: the parts' sums, weighed by their maxima, in a fixed order
// (GROUPS groups of lanes, every GROUPS-th part each, then the groups).  Latency bounds (3.5 us, of which an empty launch
// is 2); where few heads have many parts, what a CU fetches, about 35 KB a microsecond: those are cut into slices.
template <int D, int SLICES>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(AttnArgs a, Split sp) {
  constexpr int LANES = D / 4 / SLICES, GROUPS = 256 / LANES, AHEAD = 4;
  __shared__ at_f32x4 part[GROUPS][LANES];
  __shared__ float weights[kTarget + 1], totals[4];
  const int h = blockIdx.x % a.Hq, b = blockIdx.x / a.Hq;
  const int32_t* plan = (const int32_t*)(a.ws + plan_at(sp, D));
  const int size = plan[0], first = plan[1 + b], len = clamp_len(a.lens[b], a.keys);
  const int parts = (int)(((uint32_t)len + (uint32_t)size - 1) / (uint32_t)size);
  if (parts <= 1) return;
  const int head = h / sp.G, g = h % sp.G;
  auto slot = [&](int i) {
    return ((int64_t)(first + i) * sp.heads + head * sp.tiles + g / kRows) * sp.rows + g % kRows;
  };
  const float2* __restrict__ stats = (const float2*)(a.ws + stats_at(sp, D));
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES, d = (int)blockIdx.y * (D / SLICES) + 4 * l;
  at_f32x4 ahead[AHEAD];  // the first sums come while the weights are made
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) ahead[k] = *(const at_f32x4*)(a.ws + slot(min(group + k * GROUPS, parts - 1)) * D + d);
  float most = kNegInf, mine = kNegInf, sum = 0.0f;
  for (int i = threadIdx.x & 63; i < parts; i += 64) most = fmaxf(most, stats[slot(i)].x);
  most = max_xor32(max_xor16(most));
#pragma unroll
  for (int x = 1; x < 16; x *= 2) most = fmaxf(most, __shfl_xor(most, x));
  for (int i = threadIdx.x; i < parts; i += 256) {
    const float2 v = stats[slot(i)];
    weights[i] = mine = part_weight(v.x, most);
    sum += mine * v.y;
  }
  sum = sum_xor32(sum_xor16(sum));
#pragma unroll
  for (int x = 1; x < 16; x *= 2) sum += __shfl_xor(sum, x);
  if ((threadIdx.x & 63) == 0) totals[threadIdx.x >> 6] = sum;
  __syncthreads();
  at_f32x4 y{0, 0, 0, 0};
  auto add = [&](const at_f32x4& v, float f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += f * v[j];
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (group + k * GROUPS < parts) add(ahead[k], weights[group + k * GROUPS]);
#pragma unroll 4
  for (int i = group + AHEAD * GROUPS; i < parts; i += GROUPS) add(*(const at_f32x4*)(a.ws + slot(i) * D + d), weights[i]);
  part[group][l] = y;
  __syncthreads();
  if (group) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += part[i][l][j];
  }
  const float total = (totals[0] + totals[1]) + (totals[2] + totals[3]);
  const float inv = total == 0.0f ? 0.0f : (a.kv.v_scale ? a.kv.v_scale[head] : 1.0f) / total;
  *(u32x2_t*)(a.out + ((int64_t)b * a.Hq + h) * D + d) =
      u32x2_t{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
}

template <int D>
void launch(const AttnArgs& a, const Split& sp, hipStream_t stream) {
  const bool split = may_split(a.keys);
  const uint32_t units = (uint32_t)(split ? sp.units : (int64_t)a.B * sp.heads);
  auto* kernel = a.kv.f8 ? (split ? attn_decode_kernel<D, true, true> : attn_decode_kernel<D, true, false>)
                         : (split ? attn_decode_kernel<D, false, true> : attn_decode_kernel<D, false, false>);
  kernel<<<units, 64 * kWaves, 0, stream>>>(a, sp);
  if (!split) return;
  const uint32_t rows = (uint32_t)(a.B * a.Hq);
  // four slices: one token, 40 over 8 heads, 131072 keys 88.4 -> 87.5 us, 32 over one 40.7 -> 37.1; but 1000 keys,
  // 32 over 8 heads, 8.2 -> 8.5, and 64 ragged sequences 55.3 -> 62.2
  if (rows < 256 && a.keys > 16384) attn_decode_join_kernel<D, 4><<<dim3(rows, 4), 256, 0, stream>>>(a, sp);
  else attn_decode_join_kernel<D, 1><<<rows, 256, 0, stream>>>(a, sp);
}

}  // namespace

size_t attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys) {
  const Split sp = split_of(B, Hq, Hkv);
  return may_split(keys) ? (size_t)(plan_at(sp, (int)D) + 1 + B) * sizeof(float) : 0;
}

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t stream) {
  const Split sp = split_of(a.B, a.Hq, a.kv.heads);
  if (a.kv.dim == 64) launch<64>(a, sp, stream);
  else launch<128>(a, sp, stream);
  return hipGetLastError();
}

}  // namespace ql
