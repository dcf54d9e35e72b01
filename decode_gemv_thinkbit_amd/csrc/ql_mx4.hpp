// Device helpers for microscaled 4-bit floats (MX4), shared by the kernels that read them.
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

// 16 bytes at p (global memory)
__device__ __forceinline__ u32x4_t ld_b128(const void* p) { return *(gu32x4p)p; }
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
// 16 (or 4) bytes per lane: lane l's bytes land at lds + 16 l (4 l); lds is wave-uniform.  With `now`
// false nothing is read or written, but the load still counts, so waits by count stay right and no
// branch splits a loop's block.  The compiler does not see the write: readers wait with wait_vm (and a
// barrier, if other waves read).  m0 is set for each load: nothing else here keeps a value in it.
__device__ __forceinline__ void dma16(uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void dma16_if(bool now, uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\t"
               "global_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1"
               :: "s"(lds), "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(now ? ~0u : 0u)) : "memory");
}
__device__ __forceinline__ void dma4_if(bool now, uint32_t lds, const uint8_t* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\t"
               "global_load_lds_dword %1, %2\n\ts_mov_b64 exec, -1"
               :: "s"(lds), "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(now ? ~0u : 0u)) : "memory");
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
// of row r at column b ^ (r / 2 % 8); its scales are two dwords a row; a token is 512 bytes, granule g
// (eight inputs) of token m at column g ^ m.  All operand reads are then free of bank conflicts.
// DEPTH stages of the wave's own, no barrier.  The matrix instruction's lane (q, r) holds row r; token
// 4q + i of row r comes out in acc[b][t][i].
template <int NB, int R, int XP, int DEPTH>
struct Skinny {
  static constexpr int kTile = 2048 + 256;  // codes and scales of a tile
  static constexpr int kStage = NB * R * kTile + XP * 1024;
  static constexpr int kLds = DEPTH * kStage;  // per wave
  static constexpr int kLoads = NB * R * 3 + XP;
  static_assert(DEPTH * kLoads < 64, "the load counter has six bits");

  const uint8_t *codes[NB], *scales[NB], *x;
  uint32_t code_off[2 * R];  // the lane's row and block of each piece
  uint32_t scale_off[R];     // the lane's row
  uint32_t x_off[XP];        // the lane's token and granule
  int block[2], gran[XP];

  // row(t, i): byte-row index (already clamped to the matrix) of row i of tile t; token(m): row index of x
  template <class Row, class Token>
  __device__ __forceinline__ void init(int K, Row row, Token token) {
    const int lane = threadIdx.x & 63;
    const uint32_t row_bytes = (uint32_t)K / 2, stride = (uint32_t)mx4_scale_stride(K);
#pragma unroll
    for (int h = 0; h < 2; ++h) block[h] = (lane & 7) ^ (4 * h + (lane >> 4));
#pragma unroll
    for (int t = 0; t < R; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) code_off[2 * t + h] = (uint32_t)row(t, 8 * h + (lane >> 3)) * row_bytes + block[h] * 16;
      scale_off[t] = (uint32_t)row(t, (lane >> 1) & 15) * stride;
    }
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int m = 2 * i + (lane >> 5);
      gran[i] = (lane & 31) ^ (m & 15);
      x_off[i] = (uint32_t)token(m) * (uint32_t)K * 2 + gran[i] * 16;
    }
  }

  template <bool TAIL>
  __device__ __forceinline__ void send(bool now, uint32_t lds, int K, int p) const {
    const int lane = threadIdx.x & 63, nblk = K / kMxBlock, nchunk = (nblk + 3) / 4;
    uint32_t at = lds;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < R; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t back = TAIL ? (uint32_t)max(0, 8 * p + block[h] - (nblk - 1)) * 16 : 0u;
          dma16_if(now, at + 1024 * h, codes[b] + (int64_t)p * 128, code_off[2 * t + h] - back);
        }
        dma4_if(now, at + 2048, scales[b], scale_off[t] + (uint32_t)min(2 * p + (lane & 1), nchunk - 1) * 4);
        at += kTile;
      }
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const uint32_t back = TAIL ? (uint32_t)max(0, 32 * p + gran[i] - (K / 8 - 1)) * 16 : 0u;
      dma16_if(now, at, x + (int64_t)p * 512, x_off[i] - back);
      at += 1024;
    }
  }

  // smem: the wave's kLds bytes
  template <bool TAIL>
  __device__ __forceinline__ void run(f32x4_t (&acc)[NB][R], const uint8_t* smem, int K, int first, int step) const {
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    const int nblk = K / kMxBlock, npair = (nblk + 7) / 8;
    const uint32_t lds = lds_offset(smem);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) send<TAIL>(first + d * step < npair, lds + d * kStage, K, min(first + d * step, npair - 1));
    int d = 0;
    for (int p = first; p < npair; p += step) {
      wait_vm<(DEPTH - 1) * kLoads>();
      const uint8_t* st = smem + d * kStage;
      u32x4_t w[NB][R][2], a[2][4];
      u32x2_t s[NB][R];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const uint8_t* tile = st + (b * R + t) * kTile;
          s[b][t] = *reinterpret_cast<const u32x2_t*>(tile + 2048 + r * 8);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            w[b][t][h] = *reinterpret_cast<const u32x4_t*>(tile + r * 128 + (((4 * h + q) ^ (r >> 1)) << 4));
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[h][j] = *reinterpret_cast<const u32x4_t*>(st + NB * R * kTile + (r < 2 * XP ? r : 0) * 512 +
                                                     (((16 * h + 4 * q + j) ^ (r < 2 * XP ? r : 0)) << 4));
      wait_lgkm();  // the stage is read: send into it
      send<TAIL>(p + DEPTH * step < npair, lds + d * kStage, K, min(p + DEPTH * step, npair - 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = !TAIL || 8 * p + 4 * h + q < nblk;  // blocks past K: zeros
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (TAIL) a[h][j] = in ? a[h][j] : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int t = 0; t < R; ++t) {
            if (TAIL) w[b][t][h] = in ? w[b][t][h] : u32x4_t{0u, 0u, 0u, 0u};
            const float scale = in ? mx4_scale_f32((s[b][t][h] >> (8 * q)) & 255u) : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][t] = mfma_bf16(a[h][j], mx4_bf16x8(w[b][t][h][j], scale), acc[b][t]);
          }
      }
      d = d + 1 == DEPTH ? 0 : d + 1;
    }
    wait_vm<0>();  // nothing may land in LDS after this
  }
};

}  // namespace ql
