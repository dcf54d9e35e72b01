// Microscaled 4-bit floats (MX4): device helpers shared by the kernels that read them, and the launchers.
//
// A value is e2m1(code) * 2^(s - 127): code bits are sign, two of exponent, one of mantissa
// (0, 0.5, 1, 1.5, 2, 3, 4, 6), and one byte s is shared by 32 consecutive inputs of a row.  A
// block of 32 codes is 16 bytes, so one 128-bit load holds exactly one block of one row and one
// scale; a "chunk" is 128 inputs (four blocks, and the aligned dword of their four scales).
//
// Both matrix instructions used here take their operands as lane (q, r) = (lane / 16, lane % 16)
// holding row r, block q of a chunk:
//  - v_mfma_scale_f32_16x16x128_f8f6f4 reads the block's codes and scale byte as they are stored;
//  - v_mfma_f32_16x16x32_bf16 takes eight inputs per lane; instruction j of a chunk takes codes
//    8j .. 8j+7 of every lane's block, so its 32 inputs are 128c + 32q + 8j .. +7 over q (the
//    order of a sum's terms is free as long as both operands use it).
// The bf16 operands are exact: a code times a power of two keeps two significant bits, bf16 has
// fp32's exponent range, and its subnormals (s = 0) are multiplied, not flushed.  s = 255 is NaN.
#pragma once

#include "ql_internal.hpp"
#include "ql_stream.hpp"

namespace ql {

constexpr int kMxBlock = 32;   // inputs per scale
constexpr int kMxChunk = 128;  // inputs per chunk: four blocks

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

typedef const __attribute__((address_space(1))) uint32_t* mx_gu32p;

__host__ __device__ inline int64_t mx4_scale_stride(int64_t K) { return (K + kMxChunk - 1) / kMxChunk * 4; }

// 16 or 4 bytes at p (global memory)
__device__ __forceinline__ u32x4_t ld_b128_nt(const void* p) { return __builtin_nontemporal_load((gu32x4p)p); }
__device__ __forceinline__ uint32_t ld_b32(const void* p) { return *(mx_gu32p)p; }

// 2^(s - 127) as the conversions take it: the byte as a float's exponent (0 means 2^-127 to them)
__device__ __forceinline__ float mx4_scale_f32(uint32_t s) { return __uint_as_float(s << 23); }

// The eight codes of one dword times 2^(s - 127), as bf16 (exact)
__device__ __forceinline__ bf16x8_t mx4_bf16x8(uint32_t w, float scale) {
  u32x4_t v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(bf16x8_t, v);
}

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- loads straight into LDS
// 16 (or 4) bytes per lane: lane l's bytes land at lds + 16 l (4 l); lds is wave-uniform.  The compiler
// does not see the write: readers wait with wait_vm (and a barrier, if other waves read).  m0 is set in
// each block: nothing else here keeps a value in it.  Wait states the compiler does not count inside these
// blocks: one between a write of m0 and the load, five between a vector instruction's write of a scalar
// register (a lane read of an address) and a load that uses it.

__device__ __forceinline__ void dma16(uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform_ptr(base)) : "memory");
}
// The same for an address and a base that scalar instructions made (a test reads the assembly for it)
__device__ __forceinline__ void dma16_scalar(uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(off), "s"(base) : "memory");
}
// With `now` false nothing is read or written, but the load still counts, so waits by count stay right and
// no branch splits a loop's block.
__device__ __forceinline__ void dma16_if(bool now, uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\ts_nop 1\n\t"
               "global_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform_ptr(base)),
                  "s"(__builtin_amdgcn_readfirstlane(now ? ~0u : 0u)) : "memory");
}
// Two pieces, to lds and lds + 1024, from base + 1024 + off0 and base + 1024 + off1 (an instruction's
// offset moves both of its addresses).
__device__ __forceinline__ void dma16_two(uint32_t lds, const uint8_t* base, uint32_t off0_plus_1024, uint32_t off1) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %3\n\t"
               "global_load_lds_dwordx4 %2, %3 offset:1024"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off0_plus_1024), "v"(off1), "s"(uniform_ptr(base)) : "memory");
}
__device__ __forceinline__ void dma4(uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dword %1, %2"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform_ptr(base)) : "memory");
}
__device__ __forceinline__ void dma4(uint32_t lds, const uint8_t* p) {  // p per lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}
__device__ __forceinline__ void wait_lgkm() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// ---------------------------------------------------------------- a few tokens times 16-row tiles
// A wave multiplies R tiles of 16 rows of each of NB matrices by up to 2 XP tokens (at most 16), over
// pairs of chunks first, first + step, ... .  A pair (256 inputs) of a tile is 128 bytes a row, whole
// cache lines: read row by row straight into LDS (a lane order that the matrix instruction could take
// from registers would touch 64 lines a load for 16 bytes each), as two pieces of eight rows, block b
// of row r at column b ^ (r / 2 % 8); a token is 512 bytes, granule g (eight inputs) of token m at
// column g ^ m.  Operand reads are then free of bank conflicts.  Scales are two dwords a row and pair:
// read for kBand pairs at a time, as every read of a pair's alone would touch as many lines as its
// codes do. One stage of the wave's own, no barrier: a pair is read into registers, the next one sent
// for, then the products are made (two stages for half as many waves were as fast or slower).  The
// matrix instruction's lane (q, r) holds row r; token 4q + i of row r comes out in acc[b][t][i].
template <int NB, int R, int XP>
struct Skinny {
  static constexpr int kTiles = NB * R, kBand = 2, kScaleLoads = kTiles * kBand / 2;
  static constexpr int kXAt = kTiles * 2048, kScalesAt = kXAt + XP * 1024;
  static constexpr int kLds = kScalesAt + kScaleLoads * 256;  // per wave
  static_assert(kTiles * 2 + kScaleLoads + XP < 64, "the load counter has six bits");
  static_assert(XP == 1 || XP % 2 == 0, "");

  const uint8_t* codes[NB];           // each 1024 below its matrix
  const uint8_t* scales[NB];
  const uint8_t* x = nullptr;         // 1024 below the tokens (XP > 1)
  uint32_t code_off[2 * R];           // the lane's row and block of each piece (the first of two + 1024)
  uint32_t scale_off[R * kBand / 2];  // the lane's row of each piece
  uint32_t x_off[XP];                 // the lane's token and granule (the first of two + 1024)
  int pieces = XP;                    // of the tokens: those past it are not loaded

  static __device__ __forceinline__ int block(int h) {
    const int lane = threadIdx.x & 63;
    return (lane & 7) ^ (4 * h + (lane >> 4));
  }
  static __device__ __forceinline__ int gran(int i) {
    const int lane = threadIdx.x & 63;
    return (lane & 31) ^ ((2 * i + (lane >> 5)) & 15);
  }
  // c[b], s[b]: the matrices (from the tiles' first row on); row(t, i): row i of tile t in them, within
  // the matrix; tokens: bf16 rows of K; token(m): the row of token slot m
  template <class Row, class Token>
  __device__ __forceinline__ void init(int K, const uint8_t* const (&c)[NB], const uint8_t* const (&s)[NB], Row row,
                                       const void* tokens, Token token) {
    const int lane = threadIdx.x & 63;
    const uint32_t row_bytes = (uint32_t)K / 2, stride = (uint32_t)mx4_scale_stride(K);
#pragma unroll
    for (int b = 0; b < NB; ++b) codes[b] = c[b] - 1024;
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        code_off[2 * t + h] = (uint32_t)row(t, 8 * h + (lane >> 3)) * row_bytes + block(h) * 16 + (h ? 0 : 1024);
#pragma unroll
    for (int b = 0; b < NB; ++b) scales[b] = s[b];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int i = 0; i < kBand / 2; ++i)
        scale_off[t * kBand / 2 + i] = (uint32_t)row(t, (i * 64 + lane) / (2 * kBand)) * stride;
    x = (const uint8_t*)tokens - (XP > 1 ? 1024 : 0);
#pragma unroll
    for (int i = 0; i < XP; ++i)
      x_off[i] = (uint32_t)token(2 * i + (lane >> 5)) * (uint32_t)K * 2 + gran(i) * 16 + (XP > 1 && i % 2 == 0 ? 1024 : 0);
  }

  // Loads pair p.  The last pair may end inside (TAIL): its blocks and granules past K repeat the last ones.
  template <bool TAIL>
  __device__ __forceinline__ void send(uint32_t lds, int K, int p) const {
    const int nblk = K / kMxBlock;
    if (!TAIL || 8 * p + 8 <= nblk) {  // uniform
      send_as(lds, p, [](int) { return 0u; }, [](int) { return 0u; });
    } else {
      send_as(lds, p, [&](int h) { return (uint32_t)max(0, 8 * p + block(h) - (nblk - 1)) * 16; },
              [&](int i) { return (uint32_t)max(0, 32 * p + gran(i) - (K / 8 - 1)) * 16; });
    }
  }
  template <class Back, class XBack>
  __device__ __forceinline__ void send_as(uint32_t lds, int p, Back back, XBack xback) const {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < R; ++t)
        dma16_two(lds + (b * R + t) * 2048, codes[b] + (int64_t)p * 128, code_off[2 * t] - back(0), code_off[2 * t + 1] - back(1));
    const uint8_t* xp = x + (int64_t)p * 512;
    if constexpr (XP == 1) dma16(lds + kXAt, xp, x_off[0] - xback(0));
#pragma unroll
    for (int i = 0; i + 1 < XP; i += 2) {
      if (i + 1 < pieces) dma16_two(lds + kXAt + i * 1024, xp, x_off[i] - xback(i), x_off[i + 1] - xback(i + 1));
      else if (i < pieces) dma16(lds + kXAt + i * 1024, xp, x_off[i] - xback(i));
    }
  }
  // Loads the scales of pairs p, p + step, ..., kBand of them; those past a row's end repeat its last dword.
  __device__ __forceinline__ void send_scales(uint32_t lds, int K, int p, int step) const {
    const int slot = threadIdx.x & (2 * kBand - 1);
    const uint32_t at = min((uint32_t)(2 * (p + (slot >> 1) * step) + (slot & 1)) * 4, (uint32_t)mx4_scale_stride(K) - 4);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < R * kBand / 2; ++i) dma4(lds + (b * R * kBand / 2 + i) * 256, scales[b], scale_off[i] + at);
  }

  // Adds pair p, whose stage is at st and whose scales are number `slot` of the band at sc, to acc; both are
  // read when `reading` is called.  xrow: the LDS row (token slot) that the lane's operand row r comes from.
  template <bool TAIL, class Read>
  static __device__ __forceinline__ void multiply(f32x4_t (&acc)[NB][R], const uint8_t* st, const uint8_t* sc, int slot,
                                                  int K, int p, int xrow, Read reading) {
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15, nblk = K / kMxBlock;
    u32x4_t w[NB][R][2], a[2][4];
    u32x2_t s[NB][R];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < R; ++t) {
        const uint8_t* tile = st + (b * R + t) * 2048;
        s[b][t] = *reinterpret_cast<const u32x2_t*>(sc + ((b * R + t) * 16 + r) * (8 * kBand) + slot * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[b][t][h] = *reinterpret_cast<const u32x4_t*>(tile + r * 128 + (((4 * h + q) ^ (r >> 1)) << 4));
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[h][j] = *reinterpret_cast<const u32x4_t*>(st + kXAt + xrow * 512 + (((16 * h + 4 * q + j) ^ (xrow & 15)) << 4));
    wait_lgkm();
    reading();
    uint32_t e[NB][R][2];  // scale bytes
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) e[b][t][h] = (s[b][t][h] >> (8 * q)) & 255u;
    if (TAIL && 8 * p + 8 > nblk) {  // blocks past K: zeros
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = 8 * p + 4 * h + q < nblk;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[h][j] = in ? a[h][j] : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int t = 0; t < R; ++t) {
            w[b][t][h] = in ? w[b][t][h] : u32x4_t{0u, 0u, 0u, 0u};
            e[b][t][h] = in ? e[b][t][h] : 127u;
          }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const float scale = mx4_scale_f32(e[b][t][h]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[b][t] = mfma_bf16(a[h][j], mx4_bf16x8(w[b][t][h][j], scale), acc[b][t]);
        }
  }

  // The wave's whole work: a run of jobs of the same K, each over pairs first, first + step, ...; the next
  // pair is under way while one is multiplied, into the next jobs too.  next(job) sets the loads up for the
  // job after the last one it set up (false: no more); done(acc) takes a job's sums, in the same order, `jobs`
  // times.
  //   smem: the wave's kLds bytes
  template <bool TAIL, class Next, class Done>
  __device__ __forceinline__ void run(const uint8_t* smem, int K, int first, int step, int xrow, int jobs, Next next,
                                      Done done) {
    const int npair = (K / kMxBlock + 7) / 8;
    const uint32_t lds = lds_offset(smem);
    bool more = first < npair && next(*this);
    int ahead = first, slot_ahead = 0;
    auto produce = [&]() __attribute__((always_inline)) {
      if (!more) return;
      if (slot_ahead == 0) send_scales(lds + kScalesAt, K, ahead, step);
      send<TAIL>(lds, K, ahead);
      ahead += step;
      slot_ahead = slot_ahead + 1 == kBand ? 0 : slot_ahead + 1;
      if (ahead >= npair) ahead = first, slot_ahead = 0, more = next(*this);
    };
    produce();
    for (int job = 0; job < jobs; ++job) {
      f32x4_t acc[NB][R];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < R; ++t) acc[b][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      for (int p = first, slot = 0; p < npair; p += step, slot = slot + 1 == kBand ? 0 : slot + 1) {
        wait_vm<0>();
        multiply<TAIL>(acc, smem, smem + kScalesAt, slot, K, p, xrow, produce);
      }
      done(acc);
    }
    wait_vm<0>();  // nothing may land in LDS after this
  }
};

// ---------------------------------------------------------------- launchers
// Declared here and not with the library's others: bench.py reports the headline GEMV's measured traffic only
// while the sources that decide it, the common header among them, are those it was measured on.
//
// ql_mx4.hip, ql_mx4_gemm.hip: row-major codes [rows][K/2] and scales
hipError_t launch_mx4_quantize(int64_t rows, int64_t K, int type, const void* W, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream);
hipError_t launch_mx4_dequant(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales, bool bf16,
                              void* out, hipStream_t stream);
// Decode GEMV: 16-row tiles per workgroup, and parts of K (over 1: sums in a workspace)
struct GemvPlan {
  int tiles, parts;
};
GemvPlan mx4_stream_plan(double token_bytes, int N, int K);
GemvPlan mx4_gemv_plan(int M, int N, int K);
hipError_t launch_mx4_gemv(const GemvPlan& g, int M, int N, int K, const uint8_t* codes, const uint8_t* scales,
                           const uint16_t* x, float* y, float* workspace, hipStream_t stream);
hipError_t launch_mx4_join(int64_t n, int parts, const float* in, float* y, hipStream_t stream);
struct GemmPlan {
  int tiles, parts;  // the streaming kernel, as in GemvPlan (tiles > 0)
  int tile;          // else which output tile
};
GemmPlan mx4_gemm_plan(int M, int N, int K);
hipError_t launch_mx4_gemm(const GemmPlan& g, int M, int N, int K, const uint8_t* xc, const uint8_t* xs,
                           const uint8_t* wc, const uint8_t* ws, float* y, float* workspace, hipStream_t stream);

// mixture of experts (ql_moe.hip)
hipError_t launch_moe_route(int64_t T, int E, int k, bool renorm, int type, const void* logits, int32_t* ids,
                            float* weights, hipStream_t stream);
struct MoeArgs {
  int32_t T, k, E, H, I;
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  const uint8_t *gate_codes, *gate_scales, *up_codes, *up_scales, *down_codes, *down_scales;
  float* y;
  void* workspace;
};
// How a call's kernels are laid out (the rules stand in ql_moe.hip; tests read this by its fields' order)
struct MoePlan {
  int xp, split, gate_waves, down_waves;
  bool one, small, join, wide;
  int64_t hidden_bytes, product_bytes;
};
MoePlan moe_plan(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I);
size_t mx4_moe_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I);
hipError_t launch_mx4_moe(const MoeArgs& a, hipStream_t stream);

}  // namespace ql
