// Causal attention of packed prompts (or chunks of them) over the paged cache.
//
// Sequence b's queries are rows starts[b] .. starts[b + 1] - 1 (n of them), its last query the last of its
// len = lens[b] cached tokens: query i sees the keys up to position len - n + i.  The G = Hq / Hkv heads of a
// kv head see the same keys, so rows of a tile are (query, head) pairs, 128 of n * G: short chunks of many
// heads fill a tile as long ones do.
//
// One pass over the keys, 64 at a time, with the running maximum and sum of the softmax (see attn_decode), on
// v_mfma_f32_32x32x16_bf16: lane (j, r) = (lane / 32, lane % 32) holds eight inputs, 8 j .. 8 j + 7 of 16, of
// row (or column) r, and rows 8 (i / 4) + 4 j + i % 4, i < 16, of column r of the result.
//  - scores of keys x rows: K is the first operand, so lane (j, r) gets row r's scores, and maxima and sums
//    of a row are those of two lanes;
//  - output of dims x rows: V, transposed, is the first operand, and the scores are the second one as they
//    are: registers 8 h .. 8 h + 7 of a 32-key tile are the 16 keys 16 h + 8 (e / 4) + 4 j + e % 4, e < 8, in
//    an order that V's transposing reads (ds_read_b64_tr_b16, four keys of a dim to a lane) follow.
// A wave has 32 rows, four waves share the keys' tiles in LDS; the next tile is sent for before one is used.  Two such
// groups may take turns at a row tile's keys; their sums are joined in LDS, as parts of split rows are through memory.
//
// 8192 tokens, 32 over 8 heads of 128: 520 .. 550 us (by the card), 1.03 PFLOP/s of what the causal mask leaves, where a
// large bf16 product reaches 1.50.  Nothing alone bounds: of 3500 cycles that 64 keys of two workgroups take on a CU, the
// matrix unit is busy 2048 and LDS as long (each wave reads all of K and V, V's transposing reads at half the rate of
// K's: 512 and 1024 cycles, and 64 KB are written), the vector unit half, and the clock follows the power: 1.7 GHz here,
// 2.4 without load.  More waves at once do not help (three workgroups a CU, with 32 keys a tile: 579 us against 559).
// Leaving out (in copies) the softmax saves 7 %, the LDS reads 22 %, the loads into LDS 12 %.  Tried and slower or equal:
// 64 rows a wave, which would halve the reads (512 registers, of which vector instructions reach half: 780 us); 256
// rows of eight waves a workgroup (540 against 535); a tile in two halves, one's softmax under the other's products
// (+ 15 us), also with a fixed order of issue (+ 30); weights made before their maximum is known (+ 15); V's operands
// read early (- 4, but e4m3 + 13); priority for a wave at its products (- 5, but short prompts + 5 %).
#include <algorithm>
#include <type_traits>

#include "ql_attn.hpp"
#include "ql_mx4.hpp"

namespace ql {
namespace {

constexpr int kTileRows = 128, kTileKeys = 64;
constexpr int kMaxSplits = 32;
constexpr float kLag = 8.0f;     // how far (in powers of two) scores may pass the maximum in use

struct PromptPlan {
  int G, splits, least;  // least: tiles of keys of a part at least
  int layer;             // row tiles of 256 workgroups
  int groups;            // of four waves
  int64_t tiles;         // row tiles of a kv head at most
};
// Two workgroups fit a CU (of heads of 64 in bf16 three, which the plan does not use): where the rows do not make that
// many, the keys are split.  A part costs its rows' sums in fp32 written and read, so parts are long but where rows are
// few (32 over 8 heads of 128: 512 tokens take 15.5 us in one part, 22.3 in two of 256 keys; 64 tokens behind 4000
// 29.3 us in parts of 128 keys, 23.0 of 256, 24.0 of 512; 4 behind 1000 16.6 in parts of 512, 13.0 of 256).
// `keys` is what a row of the table holds, not a length: behind a table much wider than the prompt most parts are empty
// (200 tokens 10.2 us, 15.0 with a table of 8192; 1024 tokens 23.9 and 33.3).
PromptPlan plan_of(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t keys) {
  PromptPlan p;
  p.G = (int)(Hq / Hkv);
  p.tiles = T * p.G / kTileRows + B;
  p.least = T * p.G <= 2 * kTileRows ? 4 : 16;
  const int64_t blocks = (T * p.G + kTileRows - 1) / kTileRows * Hkv;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({512 / blocks, keys / (p.least * kTileKeys), kMaxSplits}));
  // Where a CU gets one workgroup or little more, two groups of waves take turns at a row tile's keys.  Microseconds with
  // one group and two, 32 over 8 heads:
  //              of 128, bf16   e4m3          of 64, bf16   e4m3
  //   200 tokens  10.1   11.1   10.8   11.5    8.0    8.2    8.4    8.5
  //   300         12.1   12.7   12.9   13.6    9.4    9.6    9.9    9.9
  //   512         15.9   15.1   17.1   16.4   12.1   11.3   12.9   11.9
  //   1024        26.7   23.4   28.4   25.7   19.6   16.9   21.0   18.1
  //   1500        36.6   32.9   39.4   34.5   26.7   21.9   28.7   24.1
  //   2048        49.3   48.0   51.1   51.3   34.7   32.7   37.0   36.1
  //   3000        83.3   95.3   86.2  102.7   54.9   64.7   57.6   73.2
  //   200 behind 3000
  //               34.5   30.6   36.8   34.1   25.7   23.0   27.0   23.8
  // Joining them takes 2 us, too much for short rows and for the short parts of few rows (16 behind 16000, of 128 in bf16,
  // 29.0 and 30.0).
  const int64_t units = (T * p.G + (B - 1) * (kTileRows / 2) + kTileRows - 1) / kTileRows * Hkv * p.splits;  // about
  const bool two = p.splits > 1    ? units <= 256 && T * p.G > 2 * kTileRows
                   : units <= 256 ? T >= 300 * B
                                  : units <= 512 && T >= 1000 * B;
  p.groups = two ? 2 : 1;
  p.layer = two ? 1 << 24 : (int)std::max<int64_t>(1, 256 / (Hkv * p.splits));
  return p;
}

struct RowTile {
  int b, first, n, len, row0;  // sequence, its first row of q, queries, cached tokens, first (query, head) of the tile
};
__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return min(max(v, lo), hi); }
// Number `want` of all sequences' tiles: of 64 sequences those with the most keys first, and a sequence's last tile,
// which sees the most keys, first, so that short tiles fill the end.  Lengths are compared in steps of a quarter of a
// power of two, seven bits at a time for all lanes.  (16 chunks of 7 .. 250 tokens behind 375 .. 6000: 175 us, 204 in the
// batch's order; 13 packed sequences of 47 .. 1189 tokens 89 and 93; 60 of 1 .. 158 21.2 either way.  The longest tiles
// of all sequences first were slower: workgroups that run together then share no keys.)
// Tiles `layer` .. 2 layer - 1, the second workgroups of the CUs (of one group of waves), are taken from their end, so
// that the longest of the first and the shortest of the second share a CU (4096 tokens, 32 over 8 heads of 128: 143 us,
// 148 without, in e4m3 147 and 155; of 64 86.8 and 87.3, in e4m3 96.6 and 103).
__device__ __forceinline__ RowTile find_tile(const AttnArgs& a, int G, int want, int layer) {
  const int lane = threadIdx.x & 63;
  uint32_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = b0 + lane;
    int first = 0, n = 0, len = 0;
    if (b < a.B) {
      first = clamp_to(a.starts[b], 0, a.T);
      n = clamp_to(a.starts[b + 1], first, a.T) - first;
      len = clamp_to(a.lens[b], 0, a.keys);
    }
    uint32_t tiles = (uint32_t)(n * G + kTileRows - 1) / kTileRows;
    int rank = lane;  // of the lane's sequence in that order
    if (a.B > 1) {
      const uint32_t size = n ? (__float_as_uint((float)(len + 1)) >> 21) - (127 << 2) : 0;
      uint64_t more = 0, same = ~(uint64_t)0;
#pragma unroll
      for (int bit = 6; bit >= 0; --bit) {
        const uint64_t set = __ballot(size >> bit & 1), mine = size >> bit & 1 ? ~(uint64_t)0 : 0;
        more |= same & set & ~mine;
        same &= ~(set ^ mine);
      }
      rank = __popcll(more) + __popcll(same & (((uint64_t)1 << lane) - 1));
      tiles = __builtin_amdgcn_ds_permute(4 * rank, (int)tiles);
    }
    const uint32_t upto = before + scan_lanes(tiles);
    if (a.B <= 64 && want >= layer) {
      const int end = min(2 * layer, (int)last_lane(upto));
      if (want < end) want = layer + end - 1 - want;
    }
    const uint64_t here = __ballot((uint32_t)want < upto);
    if (here) {
      const int place = __builtin_ctzll(here), l = __builtin_ctzll(__ballot(rank == place));
      RowTile t;
      t.b = b0 + l;
      t.first = __builtin_amdgcn_readlane(first, l);
      t.n = __builtin_amdgcn_readlane(n, l);
      t.len = __builtin_amdgcn_readlane(len, l);
      t.row0 = (__builtin_amdgcn_readlane((int)upto, place) - 1 - want) * kTileRows;
      return t;
    }
    before = last_lane(upto);
  }
  return RowTile{-1, 0, 0, 0, 0};
}

// the tiles of keys of a row tile, and of one of its parts
struct Keys {
  int tiles, per;
  __device__ __forceinline__ Keys(const RowTile& t, const PromptPlan& p) {
    const int last = min((t.row0 + kTileRows - 1) / p.G, t.n - 1);
    tiles = (max(t.len - t.n + last + 1, 0) + kTileKeys - 1) / kTileKeys;
    per = max((tiles + p.splits - 1) / p.splits, p.least);
  }
  __device__ __forceinline__ int parts() const { return max(1, (tiles + per - 1) / per); }
};

// The workspace, where rows are split: [part][kv head][row][D] sums of exp2(s - m) v, then [part][kv head][row][2] m and
// sum; a row is one of the T * G (query, head) pairs.  Rows that are split fill 512 tiles at most, so this is 34 MB at
// most, however few rows a tile has.
struct Parts {
  int64_t rows;  // T * G
  int heads, splits;
  __host__ __device__ int64_t at(int head, int split, int64_t row) const { return ((int64_t)split * heads + head) * rows + row; }
  __host__ __device__ int64_t stats(int D) const { return splits * heads * rows * D; }
  __host__ __device__ int64_t size(int D) const { return splits * heads * rows * (D + 2); }
};

typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((address_space(3))) s16x4_t* ls16x4p;

// Column c (16 bytes) of a key's row lies at column c ^ swizzle in LDS.  The 64 banks hold 256 bytes, so that
// neither K's reads (a column of 16 keys at a time) nor V's (four columns of four keys) meet in one.
template <int D> __device__ __forceinline__ int swizzle_k(int key) { return D == 128 ? key & 15 : (key >> 1) & 7; }
template <int D> __device__ __forceinline__ int swizzle_v(int key) { return D == 128 ? 4 * (key & 3) : 4 * ((key >> 1) & 1); }

// A wave's 16 keys straight into LDS at lds, 1 KB a piece (an instruction's offset moves both of its addresses);
// off[i]: the lane's place in piece i.  As for the loads in ql_mx4.hpp, readers wait, and the wait states are kept here.
__device__ __forceinline__ void dma_pieces(uint32_t lds, const uint8_t* base, const uint32_t (&off)[4]) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %5\n\t"
               "global_load_lds_dwordx4 %2, %5 offset:%6\n\tglobal_load_lds_dwordx4 %3, %5 offset:2*%6\n\t"
               "global_load_lds_dwordx4 %4, %5 offset:3*%6"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]),
                  "s"(uniform_ptr(base)), "n"(1024) : "memory");
}
__device__ __forceinline__ void dma_pieces(uint32_t lds, const uint8_t* base, const uint32_t (&off)[2]) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %3\n\t"
               "global_load_lds_dwordx4 %2, %3 offset:1024"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off[0]), "v"(off[1]), "s"(uniform_ptr(base)) : "memory");
}

// One of them; nothing is read or written where `now` is 0.  Its place among other instructions is kept.
template <int OFFSET>
__device__ __forceinline__ void dma_piece(uint32_t now, uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\ts_nop 1\n\t"
               "global_load_lds_dwordx4 %1, %2 offset:%4\n\ts_mov_b64 exec, -1"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform_ptr(base)),
                  "s"(__builtin_amdgcn_readfirstlane(now)), "n"(OFFSET) : "memory");
}

template <int D, bool F8, int GROUPS>
__global__ void __launch_bounds__(256 * GROUPS, 2) attn_prompt_kernel(AttnArgs a, PromptPlan plan) {
  constexpr int ROW = 2 * D, TILE = kTileKeys * ROW;  // bytes
  constexpr int DK = D / 16, DT = D / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t all[GROUPS * 4 * TILE];  // of each group: K, V, K, V
  __shared__ uint32_t all_odd_bits[GROUPS][2][kTileKeys][DT], odd_waves[GROUPS][4];
  const int lane = threadIdx.x & 63, j = lane >> 5, r = lane & 31;
  const int group = GROUPS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
  uint8_t* smem = all + group * 4 * TILE;
  auto& odd_bits = all_odd_bits[group];
  const int Hkv = a.kv.heads, G = plan.G;
  const int split = blockIdx.x % plan.splits, unit = blockIdx.x / plan.splits, head = unit % Hkv;
  const RowTile rt = find_tile(a, G, unit / Hkv, plan.layer);
  if (rt.b < 0) return;
  const Keys keys(rt, plan);
  const int t0 = split * keys.per, t1 = min(keys.tiles, t0 + keys.per);
  if (split && t0 >= t1) return;
  const bool whole = keys.parts() == 1;

  const int32_t* __restrict__ row = a.table + rt.b * a.table_stride;
  const int shift = a.kv.page_shift;
  const uint32_t in_page = (1u << shift) - 1;
  const uint32_t lds0 = lds_offset(smem);
  // Entries of a tile's four groups of 16 keys, lane g that of group g (mod 4), read a tile ahead; wave w brings
  // group w.  A group behind the last key takes the last key's page; entries that are no page read page 0 and
  // are masked (bit g of `bad`).
  const int key_last = max(1, min(rt.len, kTileKeys * keys.tiles)) - 1;
  auto entry = [&](int t) { return row[min(t * kTileKeys + 16 * (lane & (4 * GROUPS - 1)), key_last) >> shift]; };
  int now = 0, ahead = 0;
  if (t0 < t1) now = entry(t0), ahead = entry(t0 + GROUPS);

  const int rows = rt.n * G - rt.row0;  // those of the tile, or more
  const int base_pos = rt.len - rt.n + 1;
  const int mine = min(wave * 32 + r, rows - 1) + rt.row0;
  const int query = mine / G;
  const int limit = base_pos + query;  // keys that this row sees
  const int limit_first = base_pos + min(rt.row0 + wave * 32, rt.n * G - 1) / G;
  const int limit_tile = base_pos + rt.row0 / G;
  // (a wave without rows sees none: it only brings its keys)
  const int limit_last = wave * 32 < rows ? base_pos + min(rt.row0 + wave * 32 + 31, rt.n * G - 1) / G : 0;

  u32x4_t qf[DK];
  {
    const uint16_t* p = a.q + ((int64_t)(rt.first + query) * a.Hq + (int64_t)head * G + (mine - query * G)) * D + 8 * j;
#pragma unroll
    for (int i = 0; i < DK; ++i) qf[i] = *(gu32x4p)(p + 16 * i);
  }
  const float c = a.score_scale * (a.kv.k_scale ? a.kv.k_scale[head] : 1.0f);
  const float room = room_of(rt.len, kLag);

  struct Source { const uint8_t *k, *v; int bad; };
  auto source = [&](int t, int e) {
    const int own = __builtin_amdgcn_readlane(e, 4 * group + wave);
    const int page = (uint32_t)own < (uint32_t)a.kv.pages ? own : 0;
    const int64_t off = ((((int64_t)page * Hkv + head) << shift) + ((t * kTileKeys + 16 * wave) & in_page)) * (int64_t)(F8 ? D : 2 * D);
    return Source{a.kv.k + off, a.kv.v + off, (int)(__ballot((uint32_t)e >= (uint32_t)a.kv.pages) & (GROUPS == 1 ? 15 : 255))};
  };
  // bf16: straight into LDS, 1 KB (4 or 8 keys) a piece
  constexpr int PIECES = 16 * ROW / 1024, PER = 1024 / ROW;
  // Eight of them at once keep a wave waiting, so they go out between the first products, two for four (8192 tokens
  // 557 us, then 551; 1024 26.9 and 26.2).  With heads of 64 half as many products have to hide them: at once (70.6
  // against 73.7 for 5000 tokens, 10 over 2 heads).
  constexpr bool SPREAD = !F8 && D == 128;
  uint32_t k_off[PIECES], v_off[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = lane / (64 / PER), col = lane % (64 / PER), key = PER * i + at;
    k_off[i] = at * ROW + (col ^ swizzle_k<D>(key)) * 16;
    v_off[i] = at * ROW + (col ^ swizzle_v<D>(key)) * 16;
  }
  auto send = [&](const Source& s, int buf) {
    if constexpr (!F8) {
      const uint32_t to = lds0 + buf * 2 * TILE + wave * 16 * ROW;
      dma_pieces(to, s.k, k_off);
      dma_pieces(to + TILE, s.v, v_off);
    }
  };
  // e4m3: through registers, widened on the way
  u32x4_t raw[2][F8 ? D / 64 : 1];
  auto fetch = [&](const Source& s) {
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t off = lane / 4 * D + (lane % 4 + 4 * i) * 16;
        raw[0][i] = *(gu32x4p)(s.k + off), raw[1][i] = *(gu32x4p)(s.v + off);
      }
    }
  };
  auto put = [&](int buf) {
    if constexpr (F8) {
      const int key = lane / 4;
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = 2 * (lane % 4 + 4 * i) + h;
            const u32x2_t x = bf16_of_e4m3(raw[z][i][2 * h]), y = bf16_of_e4m3(raw[z][i][2 * h + 1]);
            uint8_t* to = smem + buf * 2 * TILE + z * TILE + (wave * 16 + key) * ROW +
                          (col ^ (z ? swizzle_v<D>(key) : swizzle_k<D>(key))) * 16;
            *(u32x4_t*)to = u32x4_t{x[0], x[1], y[0], y[1]};
          }
    }
  };
  // four keys (from `key` on) of dim 32 dt + r
  auto v_part = [&](const uint8_t* v, int dt, int key0) {
    const int key = key0 + (lane & 15) / 4, d = 32 * dt + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const uint8_t* p = v + key * ROW + ((d / 8) ^ swizzle_v<D>(key)) * 16 + (d % 8) * 2;
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls16x4p)p));
  };
  auto v_frag = [&](const uint8_t* v, int dt, int cc) {
    const u32x2_t lo = v_part(v, dt, 16 * cc + 4 * j), hi = v_part(v, dt, 16 * cc + 8 + 4 * j);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  };
  auto mfma = [](const u32x4_t& x, const u32x4_t& y, at_f32x16 z) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(at_bf16x8, x), __builtin_bit_cast(at_bf16x8, y), z, 0, 0, 0);
  };

  float m = kNegInf, sum = 0.0f;
  at_f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
  uint32_t infinities[DT] = {};  // bit e: +inf to o[dt][e], 16 + e: -inf

  Source next = {};
  int bad = 0;
  if (t0 < t1) {
    next = source(t0 + group, now);
    send(next, 0);
    fetch(next);
    put(0);
    bad = next.bad;
  }
  // q has come here, not in the loop: there a wait for it would be one for the loads into LDS too
#pragma unroll
  for (int i = 0; i < DK; ++i) asm volatile("" : "+v"(qf[i]));
  for (int first = t0; first < t1; first += GROUPS) {
    const int t = first + group, buf = (first - t0) / GROUPS & 1, key0 = t * kTileKeys;
    const bool more = first + GROUPS < t1;
    const uint8_t *kt = smem + buf * 2 * TILE, *vt = kt + TILE;
    wait_vm<0>();
    wait_lgkm();
    barrier();
    const int bad_any = bad, bad_now = bad >> (4 * group) & 15;
    if (more) {
      next = source(t + GROUPS, ahead);
      if (!SPREAD || key0 >= limit_last) send(next, buf ^ 1);
      fetch(next);
      ahead = entry(first + 2 * GROUPS);
      bad = next.bad;
    }
    // 0 * inf is NaN, also where a weight is 0 because the row does not see the key, and what memory behind the
    // last key holds is anything.  So in tiles that not every row sees whole, values that are not finite are taken
    // out of V, and noted: bit d % 32 of word d / 32 of a key, for +inf, -inf and (both) NaN.
    bool odd = false;
    if ((first + GROUPS) * kTileKeys > limit_tile || bad_any) {
      const int key = threadIdx.x % 256 / DT, dt = threadIdx.x % DT;
      bool found = false;
      if (key < kTileKeys) {
        uint32_t up = 0, down = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u32x4_t* at = (u32x4_t*)(smem + buf * 2 * TILE + TILE + key * ROW + ((4 * dt + i) ^ swizzle_v<D>(key)) * 16);
          u32x4_t v = *at;
          uint32_t most = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) most = max(most, max(v[e] & 0x7FFFu, v[e] >> 16 & 0x7FFFu));
          if (most >= 0x7F80u) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t x = v[e] >> (16 * h) & 0xFFFFu;
                if ((x & 0x7FFFu) < 0x7F80u) continue;
                up |= x != 0xFF80u ? 1u << (8 * i + 2 * e + h) : 0u;
                down |= x != 0x7F80u ? 1u << (8 * i + 2 * e + h) : 0u;
                v[e] &= h ? 0x0000FFFFu : 0xFFFF0000u;
              }
            *at = v;
            found = true;
          }
        }
        odd_bits[0][key][dt] = up, odd_bits[1][key][dt] = down;
      }
      const bool any = __ballot(found) != 0;
      if (lane == 0) odd_waves[group][wave] = any;
      __syncthreads();
      odd = odd_waves[group][0] | odd_waves[group][1] | odd_waves[group][2] | odd_waves[group][3];
    }
    if (key0 < limit_last && (GROUPS == 1 || t < t1)) {
      at_f32x16 s[2];
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[z][e] = 0.0f;
      const uint32_t now = more ? ~0u : 0u, to = lds0 + (buf ^ 1) * 2 * TILE + wave * 16 * ROW;
      u32x4_t kf[2][4];  // of four products, read four ahead
      auto k_read = [&](int g) {
        const int key = 32 * (4 * g / DK) + r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          kf[g & 1][i] = *(lu32x4p)(kt + key * ROW + (((2 * (4 * g % DK + i) + j) ^ swizzle_k<D>(key)) * 16));
      };
      auto group = [&](auto of) {
        constexpr int g = of;
        if (g + 1 < DK / 2) k_read(g + 1);
        if constexpr (SPREAD && g < 2) {
          dma_piece<2048 * g>(now, to, next.k, k_off[2 * g]);
          dma_piece<2048 * g + 1024>(now, to, next.k, k_off[2 * g + 1]);
        } else if constexpr (SPREAD) {
          dma_piece<2048 * (g - 2)>(now, to + TILE, next.v, v_off[2 * (g - 2)]);
          dma_piece<2048 * (g - 2) + 1024>(now, to + TILE, next.v, v_off[2 * (g - 2) + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * g / DK] = mfma(kf[g & 1][i], qf[4 * g % DK + i], s[4 * g / DK]);
      };
      k_read(0);
      group(std::integral_constant<int, 0>{}), group(std::integral_constant<int, 1>{});
      if constexpr (DK == 8) group(std::integral_constant<int, 2>{}), group(std::integral_constant<int, 3>{});
      const bool masked = key0 + kTileKeys > limit_first || bad_now;
      if (masked) {
        int visible = limit - key0 - 4 * j;
        asm volatile("" : "+v"(visible));  // a branch: few tiles need it
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const bool sees = 32 * z + 8 * (e / 4) + e % 4 < visible && !(bad_now >> (2 * z + e / 8) & 1);
            s[z][e] = sees ? s[z][e] : kNegInf;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int e = 1; e < 32; ++e) top = fmaxf(top, s[e / 16][e % 16]);
      top = max_xor32(top) * c;
      // The maximum in use follows only when some row's scores pass it by 2^kLag (the result is the same: it
      // cancels out, and the room has place for weights of 2^kLag)
      if (__ballot(top > m + kLag)) {
        const float m_new = fmaxf(m, top), alpha = part_weight(m, m_new);
        m = m_new;
        sum *= alpha;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[i][e] *= alpha;
      }
      const float base = m == kNegInf ? 0.0f : m + room;
      u32x4_t pf[4];
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = exp2_fast(__builtin_fmaf(s[cc / 2][8 * (cc % 2) + e], c, -base));
          sum += p[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) pf[cc][e] = pack_bf16(p[2 * e], p[2 * e + 1]);
      }
#pragma unroll
      for (int cc = 0; cc < 4; ++cc)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] = mfma(v_frag(vt, dt, cc), pf[cc], o[dt]);
      if (__builtin_expect(odd, 0)) {  // which of the lane's sums what was taken out belongs to
        for (int key = 0; key < kTileKeys; ++key) {
          if (key0 + key >= limit || (bad_now >> (key / 16) & 1)) continue;
#pragma unroll
          for (int i = 0; i < 2 * DT; ++i) {
            uint32_t w = odd_bits[i % 2][key][i / 2] >> (4 * j) & 0x0F0F0F0Fu;
            w = (w | w >> 4) & 0x00FF00FFu;
            infinities[i / 2] |= ((w | w >> 8) & 0xFFFFu) << (16 * (i % 2));
          }
        }
      }
    }
    if (more) put(buf ^ 1);
  }
  wait_vm<0>();

  sum = sum_xor32(sum);
  if constexpr (GROUPS == 2) {  // the second group's sums to the first, through LDS
    const int at = threadIdx.x % 256;
    at_f32x4* sums = (at_f32x4*)(all + 4 * TILE) + wave * (4 * DT * 64) + lane;
    float* rest = (float*)(all + 2 * TILE) + at;
    __syncthreads();
    if (group) {
#pragma unroll
      for (int i = 0; i < 4 * DT; ++i) {
        const at_f32x16& x = o[i / 4];
        sums[i * 64] = at_f32x4{x[i % 4 * 4], x[i % 4 * 4 + 1], x[i % 4 * 4 + 2], x[i % 4 * 4 + 3]};
      }
      rest[0] = m, rest[256] = sum;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) rest[512 + 256 * dt] = __uint_as_float(infinities[dt]);
    }
    __syncthreads();
    if (group) return;
    const float m1 = rest[0], most = fmaxf(m, m1), f0 = part_weight(m, most), f1 = part_weight(m1, most);
    sum = f0 * sum + f1 * rest[256];
    m = most;
#pragma unroll
    for (int i = 0; i < 4 * DT; ++i) {
      const at_f32x4 x = sums[i * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i / 4][i % 4 * 4 + e] = f0 * o[i / 4][i % 4 * 4 + e] + f1 * x[e];
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) infinities[dt] |= __float_as_uint(rest[512 + 256 * dt]);
  }
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
    if (infinities[dt]) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        o[dt][e] += infinities[dt] >> e & 1 ? -kNegInf : 0.0f;
        o[dt][e] += infinities[dt] >> (16 + e) & 1 ? kNegInf : 0.0f;
      }
    }
  if (whole) {
    // Through LDS, so that rows lie in memory as they are written, 16 bytes a lane (8 bytes of 32 rows at a time,
    // straight from the registers, took 2 us a row tile: 13 packed sequences of 47 .. 1189 tokens 97 us against 93,
    // 60 of 1 .. 158 22.3 against 20.3).  Each wave has its rows' part of the buffer that all waves had left before
    // the last tile.
    constexpr int COLS = ROW / 16, AT = 64 / COLS;
    uint8_t* stage = smem + (GROUPS == 1 ? (t1 - t0) & 1 : 0) * 2 * TILE + wave * 32 * ROW;
    auto place = [&](int row, int col) { return stage + row * ROW + (col ^ (row % COLS)) * 16; };
    const float inv = sum == 0.0f ? 0.0f : (a.kv.v_scale ? a.kv.v_scale[head] : 1.0f) / sum;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *(u32x2_t*)(place(r, 4 * dt + e / 4) + 8 * j) =
            u32x2_t{pack_bf16(o[dt][e] * inv, o[dt][e + 1] * inv), pack_bf16(o[dt][e + 2] * inv, o[dt][e + 3] * inv)};
    wait_lgkm();
#pragma unroll
    for (int i = 0; i < 32 / AT; ++i) {
      const int at = AT * i + lane / COLS, col = lane % COLS, q_at = __shfl(query, at);
      const u32x4_t y = *(lu32x4p)place(at, col);
      const int in_group = rt.row0 + wave * 32 + at - q_at * G;
      if (wave * 32 + at < rows)
        *(u32x4_t*)(a.out + ((int64_t)(rt.first + q_at) * a.Hq + (int64_t)head * G + in_group) * D + 8 * col) = y;
    }
  } else if (wave * 32 + r < rows) {
    const Parts parts{(int64_t)a.T * G, Hkv, plan.splits};
    const int64_t at = parts.at(head, split, (int64_t)rt.first * G + rt.row0 + wave * 32 + r);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *(at_f32x4*)(a.ws + at * D + 32 * dt + 2 * e + 4 * j) = at_f32x4{o[dt][e], o[dt][e + 1], o[dt][e + 2], o[dt][e + 3]};
    if (j == 0) *(float2*)(a.ws + parts.stats(D) + at * 2) = make_float2(m, sum);
  }
}

// The parts' sums, weighed by their maxima, in their order: D / 4 lanes a row.
template <int D>
__global__ void __launch_bounds__(256) attn_prompt_join_kernel(AttnArgs a, PromptPlan plan) {
  constexpr int LANES = D / 4, ROWS = 256 / LANES;
  const int Hkv = a.kv.heads, G = plan.G, unit = blockIdx.x, head = unit % Hkv;
  const RowTile rt = find_tile(a, G, unit / Hkv, plan.layer);
  if (rt.b < 0) return;
  const Keys keys(rt, plan);
  const int parts = keys.parts(), l = threadIdx.x % LANES, row = blockIdx.y * ROWS + threadIdx.x / LANES;
  if (parts == 1 || row >= rt.n * G - rt.row0) return;
  const Parts held{(int64_t)a.T * G, Hkv, plan.splits};
  const float* __restrict__ stats = a.ws + held.stats(D);
  auto slot = [&](int s) { return held.at(head, s, (int64_t)rt.first * G + rt.row0 + row); };
  // lane l of a row's has the maxima and sums of parts l, LANES + l, ..., then every lane those of all
  float most = kNegInf, total = 0.0f, mine_m[kMaxSplits / LANES], mine_w[kMaxSplits / LANES];
#pragma unroll
  for (int i = 0; i < kMaxSplits / LANES; ++i) {
    const float2 v = i * LANES + l < parts ? *(const float2*)(stats + 2 * slot(i * LANES + l)) : make_float2(kNegInf, 0.0f);
    mine_m[i] = v.x, mine_w[i] = v.y;
    most = fmaxf(most, v.x);
  }
#pragma unroll
  for (int x = 1; x < LANES; x *= 2) most = fmaxf(most, __shfl_xor(most, x));
#pragma unroll
  for (int i = 0; i < kMaxSplits / LANES; ++i) {
    const float f = i * LANES + l < parts ? part_weight(mine_m[i], most) : 0.0f;
    total += f * mine_w[i];
    mine_w[i] = f;
  }
#pragma unroll
  for (int x = 1; x < LANES; x *= 2) total += __shfl_xor(total, x);
  at_f32x4 y{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kMaxSplits / LANES; ++i) {
#pragma unroll 8
    for (int s = i * LANES; s < min(parts, (i + 1) * LANES); ++s) {
      const at_f32x4 v = *(const at_f32x4*)(a.ws + slot(s) * D + 4 * l);
      const float f = __shfl(mine_w[i], s % LANES, LANES);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += f * v[e];
    }
  }
  const float inv = total == 0.0f ? 0.0f : (a.kv.v_scale ? a.kv.v_scale[head] : 1.0f) / total;
  const int query = (rt.row0 + row) / G, in_group = rt.row0 + row - query * G;
  *(u32x2_t*)(a.out + ((int64_t)(rt.first + query) * a.Hq + (int64_t)head * G + in_group) * D + 4 * l) =
      u32x2_t{pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
}

template <int D>
void launch(const AttnArgs& a, const PromptPlan& p, hipStream_t stream) {
  const uint32_t blocks = (uint32_t)(p.tiles * a.kv.heads);
  auto run = [&](auto f8) {
    if (p.groups == 2) attn_prompt_kernel<D, f8, 2><<<blocks * p.splits, 512, 0, stream>>>(a, p);
    else attn_prompt_kernel<D, f8, 1><<<blocks * p.splits, 256, 0, stream>>>(a, p);
  };
  if (a.kv.f8) run(std::true_type{});
  else run(std::false_type{});
  if (p.splits > 1) attn_prompt_join_kernel<D><<<dim3(blocks, kTileRows * D / 1024), 256, 0, stream>>>(a, p);
}

}  // namespace

size_t attn_prompt_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t keys) {
  const PromptPlan p = plan_of(T, B, Hq, Hkv, keys);
  return p.splits > 1 ? (size_t)Parts{T * p.G, (int)Hkv, p.splits}.size((int)D) * sizeof(float) : 0;
}
int64_t attn_prompt_blocks(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t, int64_t keys) {
  const PromptPlan p = plan_of(T, B, Hq, Hkv, keys);
  return p.tiles * Hkv * p.splits;
}

hipError_t launch_attn_prompt(const AttnArgs& a, hipStream_t stream) {
  const PromptPlan p = plan_of(a.T, a.B, a.Hq, a.kv.heads, a.keys);
  if (a.kv.dim == 64) launch<64>(a, p, stream);
  else launch<128>(a, p, stream);
  return hipGetLastError();
}

}  // namespace ql
