// fp8 (e4m3) GEMM with one fp32 scale per 128 consecutive k of an activation
// row and per 128 x 128 tile of the weights: the 8-bit floating point
// counterpart of the block-scale W8A8 GEMM (StartLux-Prism README, "Why
// StartLux-Prism": a row's result does not depend on what it is batched with).
//
// Per output and block b: P_b = sum q w over the block's 128 products, then
//   f = fmaf(P_b, s_a[b][m] * s_w[n / 128][b], f)   for b ascending from f = 0,
// and y = f rounded once.  P_b comes from the matrix cores started at zero, in
// every kernel by the same instructions on the same k of each lane, so all
// kernels give a row the same bits.
//
// Which instructions depends on y's type.  v_mfma_f32_16x16x128_f8f6f4 aligns
// each eight products of consecutive k to the largest exponent among them and
// cuts what lies 2^-13 below it (found on MI355X with one large product and
// seven small ones at every place).  So products of one sign lose at most 7 *
// 2^-13 = 2^-10.2 of their sum, less than a bf16 y's rounding (2^-9 to 2^-8)
// but more than an f16 y's (2^-12 to 2^-11), and where products cancel the error
// reaches 112 * 2^-13 = 2^-6.2 of the block's largest (2^-6.4 seen; over N(0, 1)
// operands 2^-10.9, 2-norm 1.4e-5; with one activation per block 50 times the
// others 3.8e-5).  bf16 outputs take that instruction.  fp32 and f16 outputs take
// four v_mfma_f32_16x16x32_f16 on the codes converted to f16 in registers: every
// e4m3 value and product is exact there, and the error is that of fp32 sums
// (2-norm 1e-8), at half the matrix rate.
//
// Lane layout (both): lane l supplies row l % 16 of either operand; its 32
// codes of a block are the two 16-byte chunks l / 16 and l / 16 + 4.  The
// weights are the instructions' A operand, so result register r of lane l is
// weight row 4 (l / 16) + r, activation row l % 16.
//
// Times in this file are those of calls back to back.  Single ones are with
// inputs rotated through 0.6 GB or more unless they say otherwise; forms that
// are compared were timed in one run.  Traced one launch at a time, large products take 5 to 10% longer
// (8192 x 5120 x 5120: bf16 191 and 203 us, fp32 380 and 404).
#include "fp8_math.h"
#include "lds_copy.h"
#include "wave.h"

namespace prism {
namespace {

using tiled::kOutOfRange;
using tiled::make_rsrc;
using fp8::kBlock;

typedef int v8i __attribute__((ext_vector_type(8)));

// Workgroup barrier that the compiler may not move memory accesses across.
__device__ inline void barrier() { asm volatile("s_barrier" ::: "memory"); }

// f rounded to an output.  f is opaque here: the compiler would otherwise make
// one instruction of the last fma and the rounding to fp16, without the fp32
// rounding between them, in some kernels and not in others.
template <typename OUT>
__device__ inline OUT rounded(float f) {
  asm("" : "+v"(f));
  return (OUT)f;
}

// s_waitcnt lgkmcnt(0), no wait on vmcnt or expcnt (gfx9 encoding).
__device__ inline void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// v as a value the compiler knows nothing about: what is computed from it is
// computed at each use, not held in registers over the loop.
__device__ inline uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ inline float uniform(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// Workgroup b of n -> its place in a list of n tiles: each of the 8 XCDs, which
// receive workgroups in turn, takes a contiguous range.
__device__ inline int xcd_order(int b, int n) {
  const int xcd = b % 8, base = n / 8, rem = n % 8;
  return xcd * base + min(xcd, rem) + b / 8;
}

// Tile `id`: groups of 8 tile rows, column by column, so that neighbouring
// tiles, which run together on an XCD, share operand panels in its L2.
__device__ inline void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kGroup = 8;
  const int per_group = kGroup * tiles_n;
  const int grp = id / per_group, first = grp * kGroup;
  const int gm = min(tiles_m - first, kGroup);
  const int in = id - grp * per_group;
  tm = first + in % gm;
  tn = in / gm;
}

// Codes of a lane to f16, eight consecutive ones per operand.
__device__ inline fp8::v8h to_f16(const v4i c, int hi) {
  fp8::v8h o;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * hi + d], 1.0f, false);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)c[2 * hi + d], 1.0f, true);
    o[4 * d] = a[0];
    o[4 * d + 1] = a[1];
    o[4 * d + 2] = b[0];
    o[4 * d + 3] = b[1];
  }
  return o;
}

// 16 x 16 tiles: a lane's chunks l / 16 and l / 16 + 4 of its row's block.
struct Frag16 {
  v4i c[2];
};

template <bool EXACT>
struct Operand16;

template <>
struct Operand16<false> {
  v8i v;
  Operand16() = default;
  __device__ inline explicit Operand16(const Frag16& f)
      : v{f.c[0][0], f.c[0][1], f.c[0][2], f.c[0][3], f.c[1][0], f.c[1][1], f.c[1][2], f.c[1][3]} {}
};

template <>
struct Operand16<true> {
  fp8::v8h v[4];
  Operand16() = default;
  __device__ inline explicit Operand16(const Frag16& f) {
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = to_f16(f.c[s / 2], s % 2);
  }
};

__device__ inline v4f block_sum(const Operand16<false>& a, const Operand16<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ inline v4f block_sum(const Operand16<true>& a, const Operand16<true>& b) {
  v4f p{0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[s], b.v[s], p, 0, 0, 0);
  return p;
}

// Few rows (M <= 16 MT): bound by reading the weights once.  A workgroup owns
// 16 CB columns and its waves share out K: the chain over the blocks cannot be
// split, but the blocks' sums can.  In rounds of WAVES blocks, each wave
// multiplies its block straight from global memory (a lane's operands are
// two 16-byte loads per row tile and block; those of the next round are
// issued before this one's are used) and leaves the sums in LDS with the
// blocks' scales s_a s_w; after one barrier, threads fold the round's blocks
// into their outputs in order.  Rows past RP (4 where M <= 4) are not stored.
// M = 1, 5120 x 5120, bf16: 7.3 us with weights in the cache behind the L2s, 8.4
// from HBM (26 MB: 5.2 at a large copy's rate, which 100003 x 2560 at M = 4
// nearly reaches: fp32 53 us, 4.8 TB/s).
template <typename OUT, bool EXACT, int MT, int RP, int CB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void gemm_fp8_small_kernel(const uint8_t* __restrict__ q,
                                                                    const float* __restrict__ s_a,
                                                                    const uint8_t* __restrict__ w,
                                                                    const float* __restrict__ s_w,
                                                                    OUT* __restrict__ y, int M, int N, int K) {
  static_assert(RP == 16 || (RP == 4 && MT == 1), "rows kept of a row tile");
  constexpr int NT = 64 * WAVES;
  constexpr int kTile = 16 * RP;             // sums kept of a 16 x 16 tile
  constexpr int kOut = MT * CB * kTile;      // outputs of the workgroup
  constexpr int kPer = (kOut + NT - 1) / NT; // per thread
  __shared__ __attribute__((aligned(16))) float lp[2][WAVES][kOut];
  __shared__ float ls[2][WAVES][16 * MT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16 * CB;
  const int KB = (K + kBlock - 1) / kBlock;
  const auto rx = make_rsrc(q, (int64_t)M * K);
  const auto rw = make_rsrc(w + (size_t)n0 * (size_t)K, (int64_t)(N - n0) * K);
  const float* swp = s_w + (size_t)(n0 / kBlock) * (size_t)KB;

  struct Round {
    Frag16 x[MT], w[CB];
    float sa, sw;  // lane l: the scales of row l (multiplied when used: here they would wait for all loads)
  };
  // Rows past M or N read zeros (past their buffer's end), as do chunks past K.
  auto load = [&](int b0, Round& d) __attribute__((always_inline)) {
    const int b = b0 + wave;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = b * kBlock + 16 * g + 64 * h;
      const bool in = k < K;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        d.x[i].c[h] = __builtin_amdgcn_raw_buffer_load_b128(
            rx, in && 16 * i + r < M ? (uint32_t)((16 * i + r) * K + k) : kOutOfRange, 0, 0);
#pragma unroll
      for (int j = 0; j < CB; ++j)
        d.w[j].c[h] =
            __builtin_amdgcn_raw_buffer_load_b128(rw, in ? (uint32_t)((16 * j + r) * K + k) : kOutOfRange, 0, 0);
    }
    const int bb = b < KB ? b : KB - 1;  // blocks past K are not folded
    d.sa = s_a[(size_t)bb * (size_t)M + (lane < M ? lane : M - 1)];
    d.sw = swp[bb];
  };
  auto multiply = [&](int buf, const Round& d) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const Operand16<EXACT> xo(d.x[i]);
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const v4f v = block_sum(Operand16<EXACT>(d.w[j]), xo);
        if (r < RP) *reinterpret_cast<v4f*>(&lp[buf][wave][(i * CB + j) * kTile + (g * RP + r) * 4]) = v;
      }
    }
    if (lane < 16 * MT) ls[buf][wave][lane] = d.sa * d.sw;
  };
  float f[kPer];
#pragma unroll
  for (int o = 0; o < kPer; ++o) f[o] = 0.0f;
  auto fold = [&](int buf, int count) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < kPer; ++o) {
      const int e = (int)threadIdx.x + NT * o;
      if (e >= kOut) break;
      const int m = 16 * (e / kTile / CB) + e / 4 % RP;
      const float* pv = &lp[buf][0][e];
      const float* sv = &ls[buf][0][m];
      if (count == WAVES) {
#pragma unroll 8
        for (int b = 0; b < WAVES; ++b) f[o] = __builtin_fmaf(pv[b * kOut], sv[b * 16 * MT], f[o]);
      } else {
        for (int b = 0; b < count; ++b) f[o] = __builtin_fmaf(pv[b * kOut], sv[b * 16 * MT], f[o]);
      }
    }
  };
  Round cur, next;
  load(0, cur);
  int buf = 0;
  for (int b0 = 0; b0 < KB; b0 += WAVES) {
    load(b0 + WAVES, next);  // past K: zeros; behind a branch, the loads before it could not be awaited alone
    multiply(buf, cur);
    __syncthreads();  // also: every thread is done folding the round before last out of the other buffer
    fold(buf, KB - b0 < WAVES ? KB - b0 : WAVES);
    cur = next;
    buf ^= 1;
  }
#pragma unroll
  for (int o = 0; o < kPer; ++o) {
    const int e = (int)threadIdx.x + NT * o;
    if (e >= kOut) break;
    const int t = e / kTile, m = 16 * (t / CB) + e / 4 % RP;
    const int n = n0 + 16 * (t % CB) + 4 * (e % kTile / (4 * RP)) + e % 4;
    if (m < M && n < N) y[(size_t)m * (size_t)N + (size_t)n] = rounded<OUT>(f[o]);
  }
}

// Operands of a call.  With `check` the functions below launch nothing: they
// only say whether the grid of the kernel that they choose can be launched.
struct Call {
  const uint8_t* q;
  const float* s_a;
  const uint8_t* w;
  const float* s_w;
  void* y;
  int M, N, K;
  hipStream_t st;
  bool check;
};

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A grid has fewer than 2^32 threads.
int check_grid(int64_t groups, int threads) {
  return groups * threads <= (int64_t)UINT32_MAX ? PRISM_OK : PRISM_ERR_INVALID_ARG;
}

template <typename OUT, bool EXACT, int MT, int RP, int CB, int WAVES>
int launch_small(const Call& c) {
  const int64_t groups = ceil_div(c.N, 16 * CB);
  if (c.check) return check_grid(groups, 64 * WAVES);
  gemm_fp8_small_kernel<OUT, EXACT, MT, RP, CB, WAVES><<<(unsigned)groups, 64 * WAVES, 0, c.st>>>(
      c.q, c.s_a, c.w, c.s_w, static_cast<OUT*>(c.y), c.M, c.N, c.K);
  return launch_status();
}

// Waves and columns per workgroup by N: about 80 to 160 workgroups of eight
// waves for narrow outputs, which are short of workgroups (MI355X, M = 1, us:
// 2560 x 9728 8.4, 16 columns more 11.8; 5120 x 5120 7.3, 16 columns fewer 8.3),
// four waves and 16 columns for wide ones (9728 x 2560 6.7, eight waves 8.0).
template <typename OUT, bool EXACT>
int launch_small_rows(const Call& c) {
  const int M = c.M, N = c.N;
#define PRISM_FP8_SMALL(MT, RP, CB, WAVES) return launch_small<OUT, EXACT, MT, RP, CB, WAVES>(c)
#define PRISM_FP8_SMALL_N(MT, RP)                    \
  if (N <= 3840) PRISM_FP8_SMALL(MT, RP, 1, 8);      \
  if (N <= 8192) PRISM_FP8_SMALL(MT, RP, 2, 8);      \
  PRISM_FP8_SMALL(MT, RP, 1, 4)
  if (M <= 4) {
    PRISM_FP8_SMALL_N(1, 4);
  }
  if (M <= 16) {
    PRISM_FP8_SMALL_N(1, 16);
  }
  if (M <= 32 || !EXACT) {  // N <= 6144 from here on
    if (N <= 3840) PRISM_FP8_SMALL(2, 16, 1, 8);
    PRISM_FP8_SMALL(2, 16, 2, 8);
  }
  if constexpr (EXACT) {
    if (N <= 3840) PRISM_FP8_SMALL(4, 16, 1, 8);
    PRISM_FP8_SMALL(4, 16, 2, 8);
  }
#undef PRISM_FP8_SMALL_N
#undef PRISM_FP8_SMALL
}

// LDS-tiled kernel.  One workgroup of 2 x WN waves owns BM = 32 TM rows by BN =
// 16 TN WN columns and walks K one 128-block (a stage) at a time; a stage is
// the block's BM + BN rows of 128 codes and the rows' scales, copied directly
// into one of R LDS buffers.
//
// A lane holds four consecutive columns of one row of each 16 x 16 tile: its
// row scale is one value per 16 rows, the fold one multiplication per 16 rows
// and one fma per output, and y leaves as whole rows.  Frag row p of
// column tile j is weight row 4 TN (p / 4) + 4 j + p % 4 of the wave's 16 TN,
// which makes a lane's columns over its tiles consecutive.
//
// A wave keeps a stage's weight rows in registers and streams its TM row tiles
// past them, each read two tiles ahead.  Each MFMA is followed by the fold of
// the one kLag before it, whose result is then there without a wait.  The last
// two row tiles are multiplied together, column tile by column tile, so that
// each weight fragment's registers are free for the next stage's as early as
// possible.
//
// Two barriers per stage hand parts of the buffer back as they are read: at
// Q (before row tile QI) every wave has read the weights and the first QI + 2
// row tiles, at P (before the last two row tiles) the rest; short tiles have P
// only.  Behind each come the copies, into those parts, of the stage R later,
// between MFMAs.  They are awaited about R - 1/2 stages later, by count
// (vmcnt), so that a line that comes from HBM has that long to arrive (waits
// taken away, the kernels take the same time).
//
// What bounds the 256 x 256 form, MI355X, M = N = K = 8192 (480-510 us, 2.2
// PFLOP/s; 8192 x 5120 x 5120: 188 to 193 us, 2.25 PFLOP/s): the matrix cores are
// busy 58 to 61% of the cycles at a clock that the power limit holds at 1.9 GHz; without
// the copies it takes 423 us, without the LDS reads 416, without the folds
// 405, without either barrier 465.  Times of these parts add up rather than
// hide behind each other, because each costs clock.  Other forms measured and
// not kept: 32 x 32 x 64 MFMAs (4% slower at 8192), all copies of a stage
// issued together (265 against 225 us at 8192 x 5120 x 5120), one barrier per
// stage (4% slower), 128 x 128 tiles of four waves (twice the copies: 560 us).
//
// The smaller forms are bound by a stage's chain of copies, barrier, LDS reads
// and MFMAs, whatever R is (500 x 2560 x 9600, 160 tiles of 64 x 128: 27 to 32
// us, 36 from HBM; in one run of 32 us, without copies 21, without LDS reads 28,
// without the barrier 29, without all three 15).  The form of exact products,
// 128 x 128, is bound by the f16 MFMAs and the conversions, which share a SIMD's
// issue (8192 x 5120 x 5120, fp32 y: 370 to 380 us, MFMAs 53% busy; 305 at the
// rate of a large 16-bit library product).  Spread between the MFMAs, the conversions took 4% fewer
// cycles and the same time, at a lower clock.
template <int WN, int TM, int TN, int R>
constexpr int kTileLds = R * ((32 * TM + 16 * TN * WN) * kBlock + 128 * WN * 4);  // R stages

// Bytes of a row of codes in front of it in its cache line.
__device__ inline uint32_t line_start(const uint8_t* base, int row, int K) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(base) + (uint64_t)row * (uint64_t)K) % kBlock;
}

// The tile of BM rows from m0 and BN columns from n0.
template <typename OUT, bool EXACT, int WN, int TM, int TN, int R, bool LINES>
__device__ __attribute__((always_inline)) inline void tile_body(int8_t* lds, const uint8_t* __restrict__ q,
                                                                const float* __restrict__ s_a,
                                                                const uint8_t* __restrict__ w,
                                                                const float* __restrict__ s_w, OUT* __restrict__ y,
                                                                int M, int N, int K, int m0, int n0) {
  constexpr int NW = 2 * WN;
  constexpr int BM = 32 * TM, BN = 16 * TN * WN;
  static_assert((TN == 2 || TN == 4) && BN % (8 * NW) == 0, "column tiles");
  static_assert(TM % 2 == 0 && (NW == 8 || NW == 4), "pairs of row tiles, 4 or 8 waves");
  static_assert(64 * NW >= BM, "one scale copy per wave covers the rows");
  // 1 KiB copies (8 rows) per wave: V per pair of row tiles (64 rows), kB for
  // the weights.
  constexpr int V = 8 / NW, kB = BN / 8 / NW;
  constexpr int QI = TM >= 6 ? 2 : 0;                  // Q stands before row tile QI (TM = 2: no Q)
  constexpr bool HAS_Q = TM >= 4;
  constexpr int kPairsQ = HAS_Q ? (QI + 2) / 2 : 0;    // pairs handed back at Q
  constexpr int nQ = HAS_Q ? kB + V * kPairsQ : 0;     // copies behind Q: weights, then those pairs
  constexpr int nP = 1 + (HAS_Q ? 0 : kB) + V * (TM / 2 - kPairsQ);  // behind P: scales, the rest
  constexpr int kXBuf = BM * kBlock, kWBuf = BN * kBlock;
  constexpr int kScales = 64 * NW;  // floats per stage
  static_assert(R * (kXBuf + kWBuf + kScales * 4) == kTileLds<WN, TM, TN, R>, "LDS");
  int8_t* const lx = lds;
  int8_t* const lw = lds + R * kXBuf;
  float* const lsa = reinterpret_cast<float*>(lds + R * (kXBuf + kWBuf));

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave / WN, wn = wave % WN;
  const int r = lane & 15, g = lane >> 4;
  const int KB = (K + kBlock - 1) / kBlock;

  // 16-byte chunk c of row x lies at chunk c ^ swz(x): the 16 rows that 16
  // neighbouring lanes read at one chunk then fall into 16 different 16-byte
  // columns of a 256-byte window (two rows).
  auto swz_a = [](int row) { return (row >> 1) & 7; };
  auto swz_b = [](int row) { return ((row >> 1) & 1) | (((row >> (TN == 4 ? 4 : 3)) & 3) << 1); };
  const v4i ra = tiled::dma::rsrc_words(q + (size_t)m0 * (size_t)K, (int64_t)min(M - m0, BM) * K);
  const v4i rb = tiled::dma::rsrc_words(w + (size_t)n0 * (size_t)K, (int64_t)(N - n0) * K);
  const uint32_t lx0 = tiled::dma::lds_addr(lx), lw0 = tiled::dma::lds_addr(lw);
  const uint32_t lsa0 = tiled::dma::lds_addr(reinterpret_cast<const int8_t*>(lsa));
  // Row group rho (8 rows) of a pair of row tiles: rows 8 (rho % 4) .. of the
  // pair's 32 rows of wave row rho / 4.  This wave copies rho = wave + NW v.
  // The swizzles repeat every 16 (weights: 64) rows, so a lane's source chunk
  // is the same in all its activation copies (weights: of each parity).
  const int arow = (wave >> 2) * 16 * TM + (wave & 3) * 8;  // + 16 TM v + 32 pair
  const int brow = wave * 8;                                // + 8 NW i
  // LINES: a row starts anywhere, and what is copied of it for a stage is not
  // the stage's block but the cache line of its number, counted from the line in
  // which the row starts: one request each, where a block that begins inside a
  // line would be two.  Block b then lies in lines b and b + 1.  The start within
  // the line is that of every eighth row.
  static_assert(!LINES || (TM == 2 && TN == 2 && R >= 4), "two lines are read, R - 3 are on their way");
  const uint32_t ox = LINES ? line_start(q, m0 + (lane >> 3), K) : 0;
  const uint32_t ow = LINES ? line_start(w, n0 + (lane >> 3), K) : 0;
  // A lane's source chunk, k - 128 stage of its row (LINES: before the row's
  // start it wraps, past K like the others).  LINES: chunk c of a block, and of
  // the line that holds it, lies at chunk (c + swz) % 8 (128 x 5120 x 5104: 15.1 us,
  // at c ^ swz 15.9).
  auto source = [&](int swz, uint32_t start) __attribute__((always_inline)) {
    const int to = lane & 7;
    return LINES ? (uint32_t)((to + (int)(start / 16) - swz) & 7) * 16 - start : (uint32_t)((to ^ swz) * 16);
  };
  const uint32_t ca = source(swz_a((wave & 3) * 8 + (lane >> 3)), ox);
  const uint32_t cb0 = source(swz_b(brow + (lane >> 3)), ow);
  const uint32_t cb1 = source(swz_b(brow + 8 * NW + (lane >> 3)), ow);
  const uint32_t xoff = (uint32_t)((lane >> 3) * K) + ca, woff = (uint32_t)((lane >> 3) * K);
  // Addresses are computed at each use where registers are short, and held over
  // the loop by the short tiles (500 x 2560 x 9600 bf16 29.6 -> 27.2 us, 128 x 5120
  // x 5120 14.7 -> 13.8).
  auto each_time = [](uint32_t v) __attribute__((always_inline)) { return TM > 2 ? fresh(v) : v; };
  // Rows past M or N lie past their buffer's end and chunks past K are sent
  // there: both read zeros.
  auto copy_x = [&](int c, int b, int buf) __attribute__((always_inline)) {  // c = V pair + v
    const uint32_t ck = (uint32_t)b * kBlock;
    const int row = arow + 16 * TM * (c % V) + 32 * (c / V);
    const uint32_t in = each_time(xoff) + ((uint32_t)(row * K) + ck);
    const uint32_t o = ca + ck < (uint32_t)K ? in : kOutOfRange;
    tiled::dma::copy_to_lds(ra, lx0 + (uint32_t)(buf * kXBuf + row * kBlock), o);
  };
  auto copy_w = [&](int i, int b, int buf) __attribute__((always_inline)) {
    const uint32_t ck = (uint32_t)b * kBlock;
    const int row = brow + 8 * NW * i;
    const uint32_t cb = NW == 4 && i % 2 == 1 ? cb1 : cb0;
    const uint32_t in = each_time(woff) + cb + ((uint32_t)(row * K) + ck);
    const uint32_t o = cb + ck < (uint32_t)K ? in : kOutOfRange;
    tiled::dma::copy_to_lds(rb, lw0 + (uint32_t)(buf * kWBuf + row * kBlock), o);
  };
  auto copy_s = [&](int b, int buf) __attribute__((always_inline)) {
    const int bb = b < KB ? b : KB - 1;
    const v4i rs = tiled::dma::rsrc_words(s_a + (size_t)bb * (size_t)M + (size_t)m0,
                                          b < KB ? (int64_t)min(M - m0, BM) * 4 : 0);
    tiled::dma::copy4_to_lds(rs, lsa0 + (uint32_t)((buf * kScales + wave * 64) * 4), (uint32_t)(wave * 64 + lane) * 4u);
  };
  auto copy_behind_q = [&](int c, int b, int buf) __attribute__((always_inline)) {
    if (c < kB) copy_w(c, b, buf);
    else copy_x(c - kB, b, buf);
  };
  auto copy_behind_p = [&](int c, int b, int buf) __attribute__((always_inline)) {
    if (c == 0) copy_s(b, buf);
    else if (!HAS_Q && c <= kB) copy_w(c - 1, b, buf);
    else copy_x(c - 1 - (HAS_Q ? 0 : kB) + V * kPairsQ, b, buf);
  };

  const int xrow = wm * TM * 16 + r;
  const int wrow = wn * 16 * TN + 4 * TN * (r >> 2) + (r & 3);
  const int xat = xrow * kBlock + ((g ^ swz_a(xrow)) * 16);
  const int wat0 = wrow * kBlock + ((g ^ swz_b(wrow)) * 16);
  // LINES: of this lane's chunks g and g + 4, those past the line that the block
  // begins in are in the next buffer.
  struct Where {
    int at[2];
    bool next[2];
  };
  auto where = [&](int row, int swz, uint32_t start) __attribute__((always_inline)) {
    Where v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v.at[h] = row * kBlock + ((g + 4 * h + swz) & 7) * 16;
      v.next[h] = (int)(start / 16) + g + 4 * h >= 8;
    }
    return v;
  };
  Where xwhere, wwhere[TN];
  if constexpr (LINES) {
    xwhere = where(xrow, swz_a(xrow), line_start(q, m0 + xrow, K));
#pragma unroll
    for (int j = 0; j < TN; ++j)
      wwhere[j] = where(wrow + 4 * j, swz_b(wrow + 4 * j), line_start(w, n0 + wrow + 4 * j, K));
  }
  auto after = [](int buf) __attribute__((always_inline)) { return buf + 1 == R ? 0 : buf + 1; };
  auto read_lines = [&](const int8_t* p, int size, const Where& v, int buf) __attribute__((always_inline)) {
    const int a = buf * size, b = after(buf) * size;
    return Frag16{*reinterpret_cast<const v4i*>(p + (v.next[0] ? b : a) + v.at[0]),
                  *reinterpret_cast<const v4i*>(p + (v.next[1] ? b : a) + v.at[1])};
  };
  auto read_x = [&](int buf, int i) __attribute__((always_inline)) {
    if constexpr (LINES) return read_lines(lx + i * 16 * kBlock, kXBuf, xwhere, buf);
    const int8_t* p = lx + buf * kXBuf + i * 16 * kBlock;
    return Frag16{*reinterpret_cast<const v4i*>(p + xat), *reinterpret_cast<const v4i*>(p + (xat ^ 64))};
  };
  auto read_w = [&](int buf, int j) __attribute__((always_inline)) {
    if constexpr (LINES) return read_lines(lw, kWBuf, wwhere[j], buf);
    const int8_t* p = lw + buf * kWBuf + j * 4 * kBlock;
    const int wat = (int)each_time((uint32_t)wat0);
    return Frag16{*reinterpret_cast<const v4i*>(p + wat), *reinterpret_cast<const v4i*>(p + (wat ^ 64))};
  };
  auto read_s = [&](int buf, int i) __attribute__((always_inline)) { return lsa[buf * kScales + xrow + 16 * i]; };
  const int nb = min((n0 + wn * 16 * TN) / kBlock, (N - 1) / kBlock);
  const float* swp = s_w + (size_t)nb * (size_t)KB;

  // MFMA t of a stage: row tile tile(t) by column tile col(t).
  constexpr int kT = TN * TM, kP = TN * (TM - 2), kQ = TN * QI;
  constexpr int kPerP = (nP + 2 * TN - 1) / (2 * TN);                         // copies per MFMA
  constexpr int kPerQ = HAS_Q ? (nQ + kP - kQ - 1) / (kP > kQ ? kP - kQ : 1) : 1;
  constexpr int kLag = 3;
  // The next weight scale is loaded behind P's reads, whose wait covers it;
  // before P, P would wait for it (us: 8192 x 5120 x 5120 bf16 187 -> 181, 128 x
  // 5120 x 5120 fp32 22.1 -> 21.2).  The large fp32 tile is not held up there (768 x
  // 5120 x 5120 50.7, behind P 52.2).
  constexpr bool kLateScale = !EXACT || !HAS_Q;
  auto tile = [](int t) { return t < kP ? t / TN : TM - 2 + (t - kP) % 2; };
  auto col = [](int t) { return t < kP ? t % TN : (t - kP) / 2; };
  v4f f[kT], p[kLag];
#pragma unroll
  for (int t = 0; t < kT; ++t) f[t] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < kLag; ++t) p[t] = v4f{0, 0, 0, 0};
  Frag16 x[2];
  float sa[2];
  float sw_next = swp[0];
  float scp[2] = {0.0f, 0.0f};  // scales of the last two row tiles of the stage before
  auto fold = [&](int i, int j, const v4f& pv, float sc) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[TN * i + j][e] = __builtin_fmaf(pv[e], sc, f[TN * i + j][e]);
  };

  // Stage b in buffer buf, the next one in bufn (constants where R = 2).
  auto stage = [&](int b, const int buf, const int bufn, const Frag16* wf, Frag16* wnext) __attribute__((always_inline)) {
    // Weight scale, read a stage ahead (past a select, since a branch would
    // split the loop body) and kept scalar; -0 past K, see below.
    const float sw = uniform(b < KB ? sw_next : -0.0f);
    if (!kLateScale) sw_next = swp[min(b + 1, KB - 1)];
    Operand16<EXACT> wo[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) wo[j] = Operand16<EXACT>(wf[j]);
    Frag16 xs[TM + 2];
    float ss[TM + 2], sc[TM];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xs[i] = x[i];
      ss[i] = sa[i];
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const int i = tile(t), j = col(t);
      const v4f pn = block_sum(wo[j], Operand16<EXACT>(xs[i]));
      __builtin_amdgcn_sched_barrier(0);
      if (t == kP || (HAS_Q && t == kQ)) {
        wait_lgkm0();  // this wave's reads of what is handed back
        if (t == kP) tiled::dma::wait_vmcnt<(R - 2 - LINES) * (nQ + nP) + (HAS_Q ? nQ + nP - 1 : 0)>();
        else tiled::dma::wait_vmcnt<(R - 1) * (nQ + nP)>();
        barrier();
      }
      if (t < kP && j == 0) {
        xs[i + 2] = read_x(buf, i + 2);
        ss[i + 2] = read_s(buf, i + 2);
      }
      if (t == kP || t == kP + TN) {
        const int a = (t - kP) / TN;
        x[a] = read_x(bufn, a);
        sa[a] = read_s(bufn, a);
      }
      if (t >= kP && (t - kP) % 2 == 1) wnext[j] = read_w(bufn, j);
      if (kLateScale && t == kP + 1) sw_next = swp[min(b + 1, KB - 1)];
      if (t >= kP) {
#pragma unroll
        for (int c = (t - kP) * kPerP; c < (t - kP + 1) * kPerP; ++c)
          if (c < nP) copy_behind_p(c, b + R, buf);
      } else if (HAS_Q && t >= kQ) {
#pragma unroll
        for (int c = (t - kQ) * kPerQ; c < (t - kQ + 1) * kPerQ; ++c)
          if (c < nQ) copy_behind_q(c, b + R, buf);
      }
      __builtin_amdgcn_sched_barrier(0);
      const int tp = (t + kT - kLag) % kT, ip = tile(tp);
      if (t >= kLag && (t == kLag || (tp < kP ? tp % TN == 0 : tp - kP < 2))) sc[ip] = ss[ip] * sw;
      fold(ip, col(tp), p[0], t >= kLag ? sc[ip] : scp[tp % 2]);
#pragma unroll
      for (int e = 0; e + 1 < kLag; ++e) p[e] = p[e + 1];
      p[kLag - 1] = pn;
      __builtin_amdgcn_sched_barrier(0);
    }
    scp[0] = ss[TM - 2] * sw;
    scp[1] = ss[TM - 1] * sw;
  };
  static_assert(kLag < kT && kLag <= 2 * TN, "the folds left over are of the last two row tiles");

  static_assert(R >= 2 && (R - 1) * (nQ + nP) < 64, "vmcnt range");
#pragma unroll
  for (int b = 0; b < R; ++b) {
#pragma unroll
    for (int c = 0; c < nQ; ++c) copy_behind_q(c, b, b);
#pragma unroll
    for (int c = 0; c < nP; ++c) copy_behind_p(c, b, b);
  }
  tiled::dma::wait_vmcnt<(R - 1 - LINES) * (nQ + nP)>();
  barrier();
  Frag16 w0[TN], w1[TN];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i] = read_x(0, i);
    sa[i] = read_s(0, i);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) w0[j] = read_w(0, j);
  // Two stages per turn; a stage past K has P = +0 from zero codes and the scale
  // +0 * -0, so its fold adds -0, which leaves any f as it is: also a -0, to
  // which a negative sum below fp32 rounds and which +0 would make a +0.
  if constexpr (R == 2) {
    for (int b = 0; b < KB; b += 2) {
      stage(b, 0, 1, w0, w1);
      stage(b + 1, 1, 0, w1, w0);
    }
  } else {
    int b0 = 0, b1 = 1;
    for (int b = 0; b < KB; b += 2) {
      stage(b, b0, b1, w0, w1);
      b0 = b1 + 1 == R ? 0 : b1 + 1;
      stage(b + 1, b1, b0, w1, w0);
      b1 = b0 + 1 == R ? 0 : b0 + 1;
    }
  }
#pragma unroll
  for (int t = 0; t < kLag; ++t) fold(tile(kT - kLag + t), col(kT - kLag + t), p[t], scp[(kT - kLag + t) % 2]);
  tiled::dma::wait_vmcnt<0>();
  __syncthreads();  // every copy has landed and every wave has read its last: the buffers are free

  // A lane holds 4 TN consecutive columns of one of 16 rows.  Through LDS (its
  // wave's own part) those rows are stored whole, 16 bytes a lane: a lane's own
  // pieces would leave gaps between the lanes' (us, stored directly and so:
  // fp32 8192 x 5120 x 5120 403 and 381, bf16 202 and 195, 5585 x 3667 x 160 39
  // and 23, bf16 27 and 18).  Rows of y start anywhere where N is odd, so these
  // are unaligned stores (element by element the last took 78 us).
  constexpr int kVec = 16 / (int)sizeof(OUT);
  constexpr int kChunks = 16 * TN / kVec;    // of a row
  constexpr int kPitch = 16 * kChunks + 16;  // 16 more bytes against bank conflicts
  static_assert(2 * WN * 16 * kPitch <= kTileLds<WN, TM, TN, R>, "LDS of the outputs");
  int8_t* const part = lds + wave * 16 * kPitch;
  const int n = n0 + wn * 16 * TN + lane % kChunks * kVec;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int c = 0; c < 4 * TN; c += kVec) {
      OUT o[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = rounded<OUT>(f[TN * i + (c + e) / 4][e % 4]);
      __builtin_memcpy(__builtin_assume_aligned(part + r * kPitch + (4 * TN * g + c) * (int)sizeof(OUT), 16), o, 16);
    }
    wave_order();
#pragma unroll
    for (int t = 0; t < kChunks / 4; ++t) {
      const int row = lane / kChunks + t * (64 / kChunks);
      const int m = m0 + (wm * TM + i) * 16 + row;
      OUT o[kVec];
      __builtin_memcpy(o, __builtin_assume_aligned(part + row * kPitch + lane % kChunks * 16, 16), 16);
      if (m >= M) continue;
      OUT* yr = y + (size_t)m * (size_t)N;
      if (n + kVec <= N) {
        __builtin_memcpy(yr + n, o, 16);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (n + e < N) yr[n + e] = o[e];
      }
    }
    wave_order();
  }
}

// One workgroup per tile, the last tiles in smaller ones: `full` tiles of 32 TM
// rows, then the others cut into TM / TAIL pieces of 32 TAIL rows each.  A
// launch whose tiles do not fill its last round of compute units takes a whole
// round for them otherwise (2048 x 17408: 544 tiles on 256 CUs are 3 rounds,
// 512 and 32 x 4 quarters little more than 2).
template <typename OUT, bool EXACT, int WN, int TM, int TN, int R, int TAIL, int RT, int OCC, bool LINES>
__global__ __launch_bounds__(128 * WN, OCC) void gemm_fp8_tile_kernel(const uint8_t* __restrict__ q,
                                                                      const float* __restrict__ s_a,
                                                                      const uint8_t* __restrict__ w,
                                                                      const float* __restrict__ s_w,
                                                                      OUT* __restrict__ y, int M, int N, int K,
                                                                      int tiles_m, int tiles_n, int full) {
  constexpr int kLds = TAIL < TM && kTileLds<WN, TAIL, TN, RT> > kTileLds<WN, TM, TN, R>
                           ? kTileLds<WN, TAIL, TN, RT>
                           : kTileLds<WN, TM, TN, R>;
  static_assert(kLds <= 160 * 1024 / OCC, "LDS");
  __shared__ __attribute__((aligned(1024))) int8_t lds[kLds];
  const int b = (int)blockIdx.x;
  if (b < full) {
    int tm, tn;
    tile_of(xcd_order(b, full), tiles_m, tiles_n, tm, tn);
    tile_body<OUT, EXACT, WN, TM, TN, R, LINES>(lds, q, s_a, w, s_w, y, M, N, K, tm * 32 * TM, tn * 16 * TN * WN);
  } else if constexpr (TAIL < TM) {
    constexpr int S = TM / TAIL;
    int tm, tn;
    const int id = xcd_order(b - full, (int)gridDim.x - full);
    tile_of(full + id / S, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * 32 * TM + id % S * 32 * TAIL;
    if (m0 < M) tile_body<OUT, EXACT, WN, TAIL, TN, RT, false>(lds, q, s_a, w, s_w, y, M, N, K, m0, tn * 16 * TN * WN);
  }
}

template <typename OUT, bool EXACT, int WN, int TM, int TN, int R, int TAIL, int RT, int OCC, bool LINES = false>
int launch_tile(const Call& c, int64_t full) {
  const int64_t tiles_m = ceil_div(c.M, 32 * TM), tiles_n = ceil_div(c.N, 16 * TN * WN);
  const int64_t groups = full + (tiles_m * tiles_n - full) * (TM / TAIL);
  if (c.check) return check_grid(groups, 128 * WN);
  gemm_fp8_tile_kernel<OUT, EXACT, WN, TM, TN, R, TAIL, RT, OCC, LINES><<<(unsigned)groups, 128 * WN, 0, c.st>>>(
      c.q, c.s_a, c.w, c.s_w, static_cast<OUT*>(c.y), c.M, c.N, c.K, (int)tiles_m, (int)tiles_n, (int)full);
  return launch_status();
}

// Number of compute units that the choices below count with (MI355X).
constexpr int kCus = 256;

// Kernel for (M, N), fitted on MI355X with up to eight sets of inputs in turn (us
// below; small operands then come from the cache behind the L2s, large ones from
// HBM; every choice gives the same bits):
//  * small kernel: M <= 8; up to 16 rows where N <= 16384 (17408 x 5120, M =
//    16: 64 x 64 tiles 20.6 against 24.0), up to 32 rows where N <= 6144 (5120
//    x 5120, M = 32: 11.9 against 15.0), for an fp32 or f16 y up to 64 rows there
//    (5120 x 5120, M = 64: 18.5 against 22.5);
//  * bf16 y: 64 x 64 tiles while they fit the CUs at once (128 x 5120 x 5120:
//    15.1, 64 x 128 tiles 18.2), 64 x 128 tiles while those do (500 x 2560 x
//    9680: 33.7, 64 x 64 40.6, 128 x 128 47), else the smallest estimate of
//    128 x 128, 192 x 256 and 256 x 256 tiles (K = 5120: 768 x 5120 32.8, 58.3
//    and 44.2; 2048 x 5120 73.6, 61.2 and 65.2; 1536 x 9728 94, 110 and 71);
//  * fp32 or f16 y, bound by the MFMAs and conversions of a wave: the smaller estimate
//    of 64 x 64 and 128 x 128 tiles (K = 5120: 1024 x 2560 42.6 and 49.7; 768 x
//    5120 58.7 and 51.6; 2048 x 5120 135 and 116).
// An estimate counts rounds of the CUs, relative to a full round of 256 x 256
// tiles, or with exact products of two 128 x 128 tiles per CU.  One workgroup per CU
// of the latter takes two thirds of the time of two; 256 x 256 tiles that fill
// at most half of their last round are cut in two there, for 0.6 of a round.
template <typename OUT, bool EXACT>
int launch(const Call& c) {
  const int M = c.M, N = c.N, K = c.K;
  auto tiles = [&](int bm, int bn) { return ceil_div(M, bm) * ceil_div(N, bn); };
#define PRISM_FP8_TILE(WN, TM, TN, R, TAIL, RT, OCC, FULL) \
  return launch_tile<OUT, EXACT, WN, TM, TN, R, TAIL, RT, OCC>(c, FULL)
  if (M <= 8 || (M <= 16 && N <= 16384) || (M <= (EXACT ? 64 : 32) && N <= 6144))
    return launch_small_rows<OUT, EXACT>(c);
  const int64_t t64 = tiles(64, 64), t128 = tiles(128, 128), rest = t128 % (2 * kCus);
  const float c128 = (float)(t128 / (2 * kCus)) + (rest == 0 ? 0.0f : rest <= kCus ? 0.66f : 1.0f);
  // Rows that do not all start on a cache line: the short tiles' own form, for
  // operands from HBM, as a model's weights are.  Sums of five shapes each, 34 to
  // 1000 rows by 640 to 9728 columns, blocks and lines (us): K = 1040 35.8 and 37.7,
  // 2064 50.5 and 49.8, 4112 78.7 and 75.2, 5104 89.9 and 86.6, 6160 122 and 112,
  // 9680 191 and 164, 14352 306 and 248; single shapes from -25% to, with few
  // columns, +12%.  Operands that stay in the cache behind the L2s lose by it: 4112
  // 57 and 67, 9680 126 and 138, 14352 209 and 211.  An exact sum is bound elsewhere
  // (fp32 128 x 5120 x 5104 21.0 and 22.4).
  const bool lines = K >= 4096 && (K % kBlock != 0 || reinterpret_cast<uintptr_t>(c.q) % kBlock != 0 ||
                                   reinterpret_cast<uintptr_t>(c.w) % kBlock != 0);
#define PRISM_FP8_SHORT(WN, OCC, FULL)                                                 \
  if (lines) return launch_tile<OUT, EXACT, WN, 2, 2, 4, 2, 4, 1, true>(c, FULL);      \
  PRISM_FP8_TILE(WN, 2, 2, 3, 2, 3, OCC, FULL)
  if constexpr (EXACT) {
    const float c64 = 0.12f + 0.165f * (float)((t64 + kCus - 1) / kCus);
    if (c64 < c128) PRISM_FP8_TILE(2, 2, 2, 3, 2, 3, 3, t64);
    PRISM_FP8_TILE(2, 4, 4, 2, 4, 2, 2, t128);
  } else {
    if (t64 <= kCus) {
      PRISM_FP8_SHORT(2, 3, t64);
    }
    if (tiles(64, 128) <= kCus) {
      PRISM_FP8_SHORT(4, 2, tiles(64, 128));
    }
    const int64_t t256 = tiles(256, 256), last = t256 % kCus;
    const float c256 = (float)(t256 / kCus) + (last == 0 ? 0.0f : 2 * last <= kCus ? 0.6f : 1.0f);
    const float c192 = 0.83f * (float)((tiles(192, 256) + kCus - 1) / kCus);
    if (0.68f * c128 < c192 && 0.68f * c128 < c256) PRISM_FP8_TILE(2, 4, 4, 2, 4, 2, 2, t128);
    if (c192 < c256) PRISM_FP8_TILE(4, 6, 4, 2, 6, 2, 1, tiles(192, 256));
    PRISM_FP8_TILE(4, 8, 4, 2, 4, 2, 1, 2 * last <= kCus ? t256 - last : t256);
  }
#undef PRISM_FP8_SHORT
#undef PRISM_FP8_TILE
}

int dispatch(const Call& c, int type) {
  if (type == PRISM_TYPE_F32) return launch<float, true>(c);
  if (type == PRISM_TYPE_F16) return launch<_Float16, true>(c);
  return launch<__bf16, false>(c);
}

}  // namespace

int check_gemm_fp8_grid(const uint8_t* q, const uint8_t* w, int type, int M, int N, int K) {
  return dispatch({q, nullptr, w, nullptr, nullptr, M, N, K, nullptr, true}, type);
}

int launch_gemm_fp8(const uint8_t* q, const float* s_a, const uint8_t* w, const float* s_w, void* y, int type, int M,
                    int N, int K, hipStream_t st) {
  return dispatch({q, s_a, w, s_w, y, M, N, K, st, false}, type);
}

}  // namespace prism
