// MX4 x MX4 GEMM: y[m][n] = sum_k X[m][k] W[n][k], both operands read as stored by the scaled matrix
// instructions (lane l of 32x32x64 holds row l % 32, block l / 32 of a 64-input step, of 16x16x128 row
// l % 16, block l / 16: 16 bytes of codes and one scale byte; products exact, sums fp32).
#include "ql_mx4.hpp"

namespace ql {
namespace {

// The scaled matrix instruction with the scale byte SEL of each operand's dword.
template <int SEL>
__device__ __forceinline__ f32x16_t mfma_mx4(u32x4_t a, u32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, SEL, (int)sa, SEL, (int)sb);
}

// WM x WN waves, (32 MT) x (32 NT) outputs each.  4096 x 12288 x K takes 26 us + 21 us per 1024 of K on random
// operands: 114 us at K = 4096, 3.6 PFLOP/s.  The fixed part are the first loads and the stores of three tiles a
// CU, while nothing else runs there (one workgroup fills its LDS).  The rest goes at 4.9 PFLOP/s, the matrix
// unit busy in 65 % of the cycles, of which there are 1.7 10^9 a second (2.3 on zeros, 6.4 PFLOP/s: the power
// sets the clock); a loop of nothing but these instructions reaches 6.5 (8.9 on zeros).  512 tokens: 20 us.
//
// A stage holds two chunks (256 inputs, a "pair") of the tile's rows: 128 bytes of codes a row, whole
// cache lines, sent as 1 KB pieces of eight rows with 16 bytes a lane.  (64 bytes a row, one chunk a
// stage, costs twice as many requests: 406 against 364 us at 4096 x 12288 x 16384.)  Lane l of a piece takes row
// l / 8 and block (l % 8) ^ (row / 2 % 8), so that one block of 16 rows sits in 16 different 16-byte
// columns of LDS: a wave's ds_read_b128 of a block of 32 rows has no bank conflict.
//
// Two stages: before the last of a pair's four half steps the next pair has landed and this one's
// fragments are all read, so one barrier per pair both publishes the one and frees the other, and the
// pieces of the pair after next have four half steps to arrive.
//
// Scales come 16 bytes a row, four chunks at once (a "quad"), in two buffers of their own; the last,
// partial quad is read with ordinary loads ahead of the loop into a third.
template <int MT, int NT, int WM, int WN>
struct Tile {
  static constexpr int kWaves = WM * WN;
  static constexpr int kM = 32 * MT * WM, kN = 32 * NT * WN;
  static constexpr int kRows = kM + kN;                 // x rows, then w rows
  static constexpr int kStage = kRows * 128;            // bytes of codes per pair
  static constexpr int kScales = kRows * 16;            // bytes of scales per quad
  static constexpr int kLds = 2 * kStage + 3 * kScales;
  static constexpr int kPieces = kRows / 8 / kWaves;    // 1 KB pieces per wave and pair
  static constexpr int kScalePieces = kRows / 64;       // 1 KB pieces of scales per quad, all waves
  static constexpr int kScaleSends = (kScalePieces + kWaves - 1) / kWaves;
  static_assert(kWaves % 2 == 0 && kRows % (8 * kWaves) == 0 && kM % 64 == 0 && kN % 64 == 0, "");
};

// TAIL: K is not a whole number of pairs; the blocks past K count as zeros.
template <int MT, int NT, int WM, int WN, bool TAIL>
__global__ void __launch_bounds__(WM * WN * 64, 2) mx4_gemm_kernel(int M, int N, int K,
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, const uint8_t* __restrict__ wc,
    const uint8_t* __restrict__ ws, float* __restrict__ y) {
  using S = Tile<MT, NT, WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S::kLds];
  constexpr int kFrags = MT + NT, kSlots = MT * NT;
  constexpr int kFirst = (S::kPieces + 1) / 2;  // sent in the last half step of a pair, the others in the next one's first
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, r = lane & 31;
  const int nblk = K / kMxBlock, nchunk = (nblk + 3) / 4, npair = (nblk + 7) / 8;
  const uint32_t row_bytes = (uint32_t)K / 2, stride = (uint32_t)mx4_scale_stride(K);
  const int across = (N + S::kN - 1) / S::kN;
  const int64_t m0 = (int64_t)(blockIdx.x / across) * S::kM, n0 = (int64_t)(blockIdx.x % across) * S::kN;
  const uint8_t* xbase = xc + m0 * row_bytes;
  const uint8_t* wbase = wc + n0 * row_bytes;
  const uint8_t* xsbase = xs + m0 * stride;
  const uint8_t* wsbase = ws + n0 * stride;
  const int mlast = (int)min((int64_t)S::kM, M - m0) - 1, nlast = (int)min((int64_t)S::kN, N - n0) - 1;

  // pieces wave, wave + kWaves, ...: x rows first.  Rows past the end repeat the last one.
  const int block = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
  uint32_t off[S::kPieces];
#pragma unroll
  for (int i = 0; i < S::kPieces; ++i) {
    const int row = (wave + S::kWaves * i) * 8 + (lane >> 3);
    const int at = row < S::kM ? min(row, mlast) : min(row - S::kM, nlast);
    off[i] = (uint32_t)at * row_bytes + block * 16;
  }
  const uint32_t lds0 = lds_offset(smem);
  // sends piece i of pair p (a pair past the last one, and the blocks of the last one past K, repeat
  // valid bytes)
  auto send_piece = [&](int p, int i) __attribute__((always_inline)) {
    const int pp = min(p, npair - 1);
    const uint32_t back = TAIL ? (uint32_t)max(0, 8 * pp + block - (nblk - 1)) * 16 : 0u;
    dma16_scalar(lds0 + (p & 1) * S::kStage + (wave + S::kWaves * i) * 1024,
          ((wave + S::kWaves * i) * 8 < S::kM ? xbase : wbase) + (int64_t)pp * 128, off[i] - back);
  };
  uint32_t scale_off[S::kScaleSends];
#pragma unroll
  for (int i = 0; i < S::kScaleSends; ++i) {
    const int row = (wave + S::kWaves * i) * 64 + lane;
    scale_off[i] = (uint32_t)(row < S::kM ? min(row, mlast) : min(row - S::kM, nlast)) * stride;
  }
  uint8_t* const sc = smem + 2 * S::kStage;
  const int full = nchunk / 4;  // full quads
  // sends the wave's pieces of quad u's scales, or nothing past the full quads
  auto send_scales = [&](int u, bool now) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::kScaleSends; ++i) {
      const int p = wave + S::kWaves * i;
      const bool is = now && u < full && ((i + 1) * S::kWaves <= S::kScalePieces || p < S::kScalePieces);
      dma16_if(is, lds0 + 2 * S::kStage + (u & 1) * S::kScales + p * 1024,
                   (p * 64 < S::kM ? xsbase : wsbase) + (int64_t)u * 16, scale_off[i]);
    }
  };
  if (nchunk & 3) {
    for (int row = threadIdx.x; row < S::kRows; row += S::kWaves * 64) {
      const uint8_t* p = (row < S::kM ? xsbase + (uint32_t)min(row, mlast) * stride
                                      : wsbase + (uint32_t)min(row - S::kM, nlast) * stride) + full * 16;
      u32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = ld_b32(p + 4 * min(j, (nchunk & 3) - 1));
      *reinterpret_cast<u32x4_t*>(sc + 2 * S::kScales + row * 16) = v;
    }
  }
  send_scales(0, true);
#pragma unroll
  for (int i = 0; i < S::kPieces; ++i) send_piece(0, i);
#pragma unroll
  for (int i = 0; i < kFirst; ++i) send_piece(1, i);

  // fragment t of half step h (0..3) of the pair in stage p & 1: the first x tile, the w tiles, the
  // other x tiles; a lane's block of half step h is 2h + half
  const int wm = wave / WN * 32 * MT, wn = S::kM + wave % WN * 32 * NT;
  const uint32_t piece = (r >> 3) * 1024 + (r & 7) * 128 + (half ^ ((r >> 1) & 7)) * 16;
  u32x4_t A[2][MT], B[2][NT];
  uint32_t sa[MT], sb[NT];
  auto read = [&](int p, int h, int t, u32x4_t(&a)[MT], u32x4_t(&b)[NT]) __attribute__((always_inline)) {
    const uint8_t* st = smem + (p & 1) * S::kStage;
    if (t == 0 || t > NT) {
      const int i = t == 0 ? 0 : t - NT;
      a[i] = *reinterpret_cast<const u32x4_t*>(st + (wm + 32 * i) * 128 + (piece ^ (h * 32)));
    } else {
      b[t - 1] = *reinterpret_cast<const u32x4_t*>(st + (wn + 32 * (t - 1)) * 128 + (piece ^ (h * 32)));
    }
  };
  // scale dword of chunk c for tile t (x tiles, then w tiles); shifted by 8 half where it is used, so that
  // nothing waits for a read: byte 2s is then the lane's own block of the chunk's half step s
  auto read_scale = [&](int c, int t) __attribute__((always_inline)) -> uint32_t {
    const uint8_t* st = sc + ((c >> 2) < full ? ((c >> 2) & 1) : 2) * S::kScales + (c & 3) * 4 + r * 16;
    return *reinterpret_cast<const uint32_t*>(st + (t < MT ? wm + 32 * t : wn + 32 * (t - MT)) * 16);
  };
  f32x16_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x16_t{};

  wait_vm<kFirst>();  // the first pair's pieces and the first quad's scales
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kFrags; ++t) read(0, 0, t, A[0], B[0]);
#pragma unroll
  for (int t = 0; t < kFrags; ++t) (t < MT ? sa[t] : sb[t - MT]) = read_scale(0, t) >> (8 * half);
  // Each matrix instruction is a slot that also issues its share of the next half step's LDS reads, of
  // the next chunk's scales and of the pieces to send, so none of them holds up the matrix unit.
  int p = 0;
  do {
    uint32_t na[MT], nb[NT];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      u32x4_t(&a)[MT] = A[h & 1];
      u32x4_t(&b)[NT] = B[h & 1];
      if (TAIL) {  // blocks past K: zero codes, scales of 1
        const bool out = 8 * p + 2 * h + half >= nblk;
        const uint32_t keep = out ? ~(0xFFu << (16 * (h & 1))) : ~0u, one = out ? 127u << (16 * (h & 1)) : 0u;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          sa[i] = (sa[i] & keep) | one;
#pragma unroll
          for (int v = 0; v < 4; ++v) a[i][v] = out ? 0u : a[i][v];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) sb[j] = (sb[j] & keep) | one;
      }
      if (h == 3) {
        // the next pair has landed and this pair's fragments are read, for this wave; after the barrier for all
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        barrier();
        sched_fence();
      }
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        f32x16_t& o = acc[t / NT][t % NT];
        o = h & 1 ? mfma_mx4<2>(a[t / NT], b[t % NT], o, sa[t / NT], sb[t % NT])
                  : mfma_mx4<0>(a[t / NT], b[t % NT], o, sa[t / NT], sb[t % NT]);
#pragma unroll
        for (int f = 0; f < kFrags; ++f) {
          if ((h & 1) && f * kSlots / kFrags / 4 == t) (f < MT ? na[f] : nb[f - MT]) = read_scale(2 * p + (h + 1) / 2, f);
          if (kSlots / 4 + f * kSlots / kFrags / 2 == t) read(h == 3 ? p + 1 : p, (h + 1) & 3, f, A[(h + 1) & 1], B[(h + 1) & 1]);
        }
        if (h == 3 && t == 0) send_scales((p >> 1) + 1, (p & 1) == 0);
#pragma unroll
        for (int i = 0; i < S::kPieces; ++i) {
          if (h == 3 && i < kFirst && i * kSlots / kFirst == t) send_piece(p + 2, i);
          if (h == 0 && i >= kFirst && (i - kFirst) * kSlots / (S::kPieces - kFirst) == t) send_piece(p + 1, i);
        }
        sched_fence();
      }
      if (h & 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i) sa[i] = na[i] >> (8 * half);
#pragma unroll
        for (int j = 0; j < NT; ++j) sb[j] = nb[j] >> (8 * half);
      }
    }
  } while (++p < npair);
  wait_vm<0>();  // nothing may land in LDS after the workgroup has ended

  // Lane (half, r) of accumulator row v holds output row 8 (v / 4) + 4 half + v % 4, column r.  Stores
  // go through a buffer resource at the row's start whose range check drops the lanes that bit 31 of
  // the offset marks as outside (rows past M, columns past N).  Non-temporal: y is not read back here
  // (118.0 against 115.8 us at 4096 x 12288 x 4096).
  const int mw = wave / WN * 32 * MT, nw = wave % WN * 32 * NT;
  uint32_t to[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    to[j] = (uint32_t)(half * 4) * (uint32_t)N * 4u + (uint32_t)(32 * j + r) * 4u + (nw + 32 * j + r <= nlast ? 0u : 0x80000000u);
  const float* yt = y + (m0 + mw) * N + n0 + nw;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int m = 32 * i + (v >> 2) * 8 + (v & 3);
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(yt + (int64_t)m * N), (short)0, 0x7FFFFFFF,
                                                          0x00020000);
      const uint32_t out = mw + m + half * 4 <= mlast ? 0u : 0x80000000u;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][v]), rsrc, to[j] | out, 0, 2);
    }
}

// Up to 64 tokens: what bounds is the stream of W, so a workgroup owns R tiles of 16 rows (as the decode
// GEMV, and with its split of K), MT tiles of 16 tokens ride along, and every wave runs whole pairs of
// chunks through an LDS stage of its own, tiles of W and of X laid out alike.  With weights from HBM 5120 x
// 5120 at 33 tokens takes 8.5 us, 28672 x 8192 at 20 34.6 (3.6 TB/s of W).
constexpr int kSkinnyWaves = 8;

template <int R, int MT, bool TAIL>
__global__ void __launch_bounds__(kSkinnyWaves * 64) mx4_gemm_skinny_kernel(int M, int N, int K,
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs, const uint8_t* __restrict__ wc,
    const uint8_t* __restrict__ ws, float* __restrict__ out) {
  constexpr int kWaves = kSkinnyWaves, kTiles = R + MT, kScaleLoads = (kTiles + 1) / 2;
  constexpr int kScaleAt = kTiles * 2048, kStage = kScaleAt + kScaleLoads * 256;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kWaves * kStage];
  static_assert(kStage >= R * MT * 1024 && 2 * kTiles + kScaleLoads < 64, "");
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nblk = K / kMxBlock, nchunk = (nblk + 3) / 4, npair = (nblk + 7) / 8;
  const uint32_t row_bytes = (uint32_t)K / 2, stride = (uint32_t)mx4_scale_stride(K);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R);
  const int last = (int)min((int64_t)16 * R, N - n0) - 1;  // rows past the end repeat the last one
  const uint8_t* wsb = ws + n0 * stride;
  // dma16_two's bases and offsets; scales of two tiles a load (lanes 0..31 an even tile, 32..63 the next)
  const uint8_t *wb = wc + n0 * row_bytes - 1024, *xb = xc - 1024;
  auto tile_row = [&](int t, int i) { return t < R ? min(16 * t + i, last) : min(16 * (t - R) + i, M - 1); };
  uint32_t code_off[2 * kTiles];
  const uint8_t* scales[kScaleLoads];
  int block[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) block[h] = (lane & 7) ^ (4 * h + (lane >> 4));
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      code_off[2 * t + h] = (uint32_t)tile_row(t, 8 * h + (lane >> 3)) * row_bytes + block[h] * 16 + (h ? 0 : 1024);
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i) {
    const int a = 2 * i, b = 2 * i + 1 < kTiles ? 2 * i + 1 : a, row = (lane >> 1) & 15;
    scales[i] = lane < 32 ? (a < R ? wsb : xs) + (uint32_t)tile_row(a, row) * stride
                          : (b < R ? wsb : xs) + (uint32_t)tile_row(b, row) * stride;
    scales[i] += (lane & 1) * 4;
  }
  const uint8_t* mine = smem + wave * kStage;
  const uint32_t lds = lds_offset(mine);
  const int step = kWaves * (int)gridDim.y, first = (int)blockIdx.y * kWaves + wave;
  auto send = [&](int p) __attribute__((always_inline)) {
    if (p >= npair) return;
    const bool tail = TAIL && 8 * p + 8 > nblk;
    uint32_t back[2] = {0u, 0u}, sback = 0u;
    if (tail) {
      back[0] = (uint32_t)max(0, 8 * p + block[0] - (nblk - 1)) * 16;
      back[1] = (uint32_t)max(0, 8 * p + block[1] - (nblk - 1)) * 16;
      sback = (uint32_t)max(0, 2 * p + (lane & 1) - (nchunk - 1)) * 4;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      dma16_two(lds + t * 2048, (t < R ? wb : xb) + (int64_t)p * 128, code_off[2 * t] - back[0], code_off[2 * t + 1] - back[1]);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) dma4(lds + kScaleAt + i * 256, scales[i] + (int64_t)p * 8 - sback);
  };
  f32x4_t acc[R][MT];
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  send(first);
  for (int p = first; p < npair; p += step) {
    wait_vm<0>();
    u32x4_t c[kTiles][2];
    u32x2_t s[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      s[t] = *reinterpret_cast<const u32x2_t*>(mine + kScaleAt + t * 128 + r * 8);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        c[t][h] = *reinterpret_cast<const u32x4_t*>(mine + t * 2048 + r * 128 + (((4 * h + q) ^ (r >> 1)) << 4));
    }
    wait_lgkm();  // the stage is read: send into it
    send(p + step);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = !TAIL || 8 * p + 4 * h + q < nblk;  // blocks past K: zero codes of W, scales of 1
      int f[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        if (TAIL && t < R) c[t][h] = in ? c[t][h] : u32x4_t{0u, 0u, 0u, 0u};
        f[t] = in ? (int)(s[t][h] >> (8 * q)) : 127;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4_t x = c[R + m][h];
        const i32x8_t A = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const i32x8_t B = {(int)c[t][h][0], (int)c[t][h][1], (int)c[t][h][2], (int)c[t][h][3], 0, 0, 0, 0};
          acc[t][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc[t][m], 4, 4, 0, f[R + m], 0, f[t]);
        }
      }
    }
  }
  wait_vm<0>();
  __syncthreads();
  f32x4_t* part = reinterpret_cast<f32x4_t*>(smem);
#pragma unroll
  for (int t = 0; t < R; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[(wave * R * MT + t * MT + m) * 64 + lane] = acc[t][m];
  __syncthreads();
  out += (int64_t)blockIdx.y * M * N;
  for (int u = wave; u < R * MT; u += kWaves) {
    f32x4_t v = part[u * 64 + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += part[(w * R * MT + u) * 64 + lane];
    const int64_t n = n0 + 16 * (u / MT) + r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = 16 * (u % MT) + 4 * q + i;
      if (m < M && n < N) out[(int64_t)m * N + n] = v[i];
    }
  }
}

template <int R, int MT>
hipError_t launch_skinny(int parts, int M, int N, int K, const uint8_t* xc, const uint8_t* xs, const uint8_t* wc,
                         const uint8_t* ws, float* out, hipStream_t stream) {
  const auto kernel = K % (2 * kMxChunk) ? mx4_gemm_skinny_kernel<R, MT, true> : mx4_gemm_skinny_kernel<R, MT, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((N + 16 * R - 1) / (16 * R)), (unsigned)parts),
                     dim3(kSkinnyWaves * 64), 0, stream, M, N, K, xc, xs, wc, ws, out);
  return hipGetLastError();
}

template <int R>
hipError_t skinny_tokens(int parts, int M, int N, int K, const uint8_t* xc, const uint8_t* xs, const uint8_t* wc,
                         const uint8_t* ws, float* out, hipStream_t stream) {
  if (M <= 16) return launch_skinny<R, 1>(parts, M, N, K, xc, xs, wc, ws, out, stream);
  if (M <= 32) return launch_skinny<R, 2>(parts, M, N, K, xc, xs, wc, ws, out, stream);
  return launch_skinny<R, 4>(parts, M, N, K, xc, xs, wc, ws, out, stream);
}

template <int MT, int NT, int WM, int WN>
hipError_t launch_tile(int M, int N, int K, const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws,
                       float* y, hipStream_t stream) {
  using S = Tile<MT, NT, WM, WN>;
  const auto kernel = K % (2 * kMxChunk) ? mx4_gemm_kernel<MT, NT, WM, WN, true> : mx4_gemm_kernel<MT, NT, WM, WN, false>;
  const int64_t tiles = ((int64_t)(N + S::kN - 1) / S::kN) * ((M + S::kM - 1) / S::kM);
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(S::kWaves * 64), 0, stream, M, N, K, xc, xs, wc, ws, y);
  return hipGetLastError();
}

}  // namespace

// Up to 64 tokens the stream of W bounds: the skinny kernel, with the decode GEMV's plan.  Above, the
// tile whose workgroups, n to a CU, take the least time: a large tile reads less per product, a small
// one spreads few outputs over more CUs.  Times of one workgroup's share of a full CU at K = 4096 (us),
// and how many such shares the latency of a CU that has few workgroups costs, both measured at
// 128 .. 4096 x 4096 .. 12288 x 4096:
GemmPlan mx4_gemm_plan(int M, int N, int K) {
  if (M <= 64) {
    const GemvPlan g = mx4_stream_plan(8.5 * (M <= 16 ? 1 : M <= 32 ? 2 : 4), N, K);
    return {g.tiles, g.parts, 0};
  }
  static const struct { int m, n; double share, least; } tiles[] = {
      {256, 256, 33.0, 1.0}, {128, 128, 11.4, 1.25}, {64, 128, 7.7, 1.5}, {64, 64, 4.9, 2.0}};
  const int64_t cus = device_cu_count();
  GemmPlan best{0, 1, 0};
  double time = 0.0;
  for (int i = 0; i < 4; ++i) {
    const int64_t groups = (int64_t)((M + tiles[i].m - 1) / tiles[i].m) * ((N + tiles[i].n - 1) / tiles[i].n);
    const double each = (double)((groups + cus - 1) / cus), t = tiles[i].share * (each > tiles[i].least ? each : tiles[i].least);
    if (i == 0 || t < time) time = t, best.tile = i;
  }
  return best;
}

hipError_t launch_mx4_gemm(const GemmPlan& g, int M, int N, int K, const uint8_t* xc, const uint8_t* xs,
                           const uint8_t* wc, const uint8_t* ws, float* y, float* workspace, hipStream_t stream) {
  if (g.tiles > 0) {
    float* out = g.parts > 1 ? workspace : y;
    const hipError_t e = g.tiles == 1   ? skinny_tokens<1>(g.parts, M, N, K, xc, xs, wc, ws, out, stream)
                         : g.tiles == 2 ? skinny_tokens<2>(g.parts, M, N, K, xc, xs, wc, ws, out, stream)
                                        : skinny_tokens<4>(g.parts, M, N, K, xc, xs, wc, ws, out, stream);
    if (e != hipSuccess || g.parts == 1) return e;
    return launch_mx4_join((int64_t)M * N, g.parts, workspace, y, stream);
  }
  if (g.tile == 0) return launch_tile<4, 2, 2, 4>(M, N, K, xc, xs, wc, ws, y, stream);
  if (g.tile == 1) return launch_tile<2, 2, 2, 2>(M, N, K, xc, xs, wc, ws, y, stream);
  if (g.tile == 2) return launch_tile<1, 2, 2, 2>(M, N, K, xc, xs, wc, ws, y, stream);
  return launch_tile<1, 1, 2, 2>(M, N, K, xc, xs, wc, ws, y, stream);
}

}  // namespace ql
