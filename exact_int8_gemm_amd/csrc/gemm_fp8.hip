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
#include "gemm_fp8_kernels.h"

namespace prism {
namespace {

using namespace fp8;

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
    tile_body<OUT, EXACT, WN, TM, TN, R, LINES>(lds, q, s_a, M, w, s_w, y, M, N, K, tm * 32 * TM, tn * 16 * TN * WN);
  } else if constexpr (TAIL < TM) {
    constexpr int S = TM / TAIL;
    int tm, tn;
    const int id = xcd_order(b - full, (int)gridDim.x - full);
    tile_of(full + id / S, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * 32 * TM + id % S * 32 * TAIL;
    if (m0 < M) tile_body<OUT, EXACT, WN, TAIL, TN, RT, false>(lds, q, s_a, M, w, s_w, y, M, N, K, m0, tn * 16 * TN * WN);
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
