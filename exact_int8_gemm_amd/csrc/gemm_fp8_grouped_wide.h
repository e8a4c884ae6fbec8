// The grouped fp8 GEMM for groups of many rows and a bf16 y: 256 columns by 256, 192
// or 128 rows a tile, in a kernel that stays on its compute unit and goes from tile to
// tile without a pause.
//
// The tile is tile_body's with eight waves and two stages: its arithmetic, its
// swizzles and its two barriers a stage are explained there.  What differs:
//  * The last two stages of a tile copy the first two of the next one, and the
//    last one reads its first operands, so that no tile waits for its first copies.
//    What is left between tiles are the conversions and stores of y (of 2560 k, 10 us
//    of 42 a tile were in front of and behind its stages).
//  * Row tile i of wave row wm is rows 32 i + 16 wm .. + 15 of the tile, so that a tile
//    of fewer rows takes the first copies of a taller one's, and all copy alike:
//    weights, rows 0 .. 63, then the row scales and the other rows.
//  * A group's rows are cut into tiles of even heights, in units of 64 rows.
//  * Workgroup s of 32 on one XCD takes every 32nd tile of a contiguous part of the
//    list, which holds a group's tiles side by side.  Where at most 16 tiles are
//    left for the last round, they are cut in two there.
//
// 32768 rows by 2560 x 2560 (430 GFLOP), us, tile_body's kernel and this one: one group
// 220 and 197 (2.18 PFLOP/s), 16 ragged ones 249 and 225, 64 ragged ones 289 and 262.  A
// stage of a tall tile takes 1.7 us, with 64 KB for each of 256 compute units, 9 to 10
// TB/s out of the L2s, and 2.5 PFLOP/s, what a large library product makes on a warm chip
// (2.4 to 3.1); that of a lower tile takes not much less (192 rows 1.4, 128 rows 1.2: 2.3 and 1.8 PFLOP/s).
// So ragged groups lose by their lower tiles, by the conversions and stores between
// tiles, and by a list that is cut into equal numbers of tiles, not into equal work;
// how much by each was not measured.  Weights from HBM add 0.4 us a stage.  Not kept: a list
// for each height, the tall tiles first, which parts a group's tiles (64 ragged groups
// 269); lines of weights touched three stages ahead (247 against 238
// with 64 even groups).
#pragma once

#include <type_traits>

#include "gemm_fp8_kernels.h"

namespace prism {
namespace fp8 {

// Operands of a grouped product.
struct Grouped {
  const uint8_t* q;
  const float* s_a;
  const int32_t* rows;     // of q, of each row of y; or null: the same one
  const int32_t* offsets;
  const uint8_t* w;
  const float* s_w;
  void* y;
  int M, R, E, N, K;       // M: rows of q, R: of y
};

// Inclusive sum over the wave's lanes.
__device__ inline int wave_inclusive(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}

// Expert e's rows lo .. hi - 1 of y.  Whatever the offsets hold, they are rows of y.
__device__ inline void rows_of(const Grouped& a, int e, int& lo, int& hi) {
  lo = e < a.E ? min(max(a.offsets[e], 0), a.R) : 0;
  hi = e < a.E ? min(max(a.offsets[e + 1], lo), a.R) : 0;
}

namespace wide {

constexpr int kRows = 256, kColumns = 256, kWaves = 8, kMaxE = 1024;
constexpr int kSlots = 32;                 // workgroups of an XCD
constexpr int kMinK = 5 * kBlock;          // three turns: a tile's row numbers have landed when they are used
constexpr int kXBuf = kRows * kBlock, kWBuf = kColumns * kBlock;
constexpr uint32_t kPast = (uint32_t)-16;  // past any buffer's end, and a constant that needs no register
constexpr int kPitch = 16 * 8 + 16;        // of a wave's 16 rows of 64 outputs
constexpr int kAtW = 2 * kXBuf, kAtScales = kAtW + 2 * kWBuf, kAtOut = kAtScales + 2 * kRows * 4;
constexpr int kAtRows = kAtOut + kWaves * 16 * kPitch, kAtTiles = kAtRows + 2 * kRows * 4;
constexpr int kLds = kAtTiles + (kMaxE + 4) * 4;
static_assert(kLds <= 160 * 1024 && kMaxE >= PRISM_EXPERTS_MAX, "LDS");

struct Tile {
  int expert, m0, rows, n0;  // rows 0: none
  int height;                // 8, 6 or 4 row tiles of a wave row
};

// Tiles that u units of 64 rows make in a column, and where tile t of n begins: the
// first u % n are one unit taller.
__device__ inline int tiles_of_units(int u) { return (u + 3) / 4; }
__device__ inline int begin_of(int t, int n, int u) { return t * (u / n) + min(t, u % n); }

// p[i] by a scalar load: i is the same in all lanes, and nothing writes there.
template <typename T>
__device__ inline T scalar(const T* p, int64_t i) {
  typedef __attribute__((address_space(4))) const T Constant;
  return reinterpret_cast<Constant*>(reinterpret_cast<uintptr_t>(p))[i];
}
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// tiled::dma's copies, wait states and all, with all but the offset in scalar registers
// as they come: made sure of by a lane read, they would first be moved to vector
// registers, and held there over the stages.  The descriptors of the codes stay in
// scalar registers; that of the scales comes from spilled ones, right in front of its
// copy.
__device__ inline void copy16(const v4i rsrc, uint32_t to, uint32_t from) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds" : "={m0}"(m0) : "s"(to), "v"(from), "s"(rsrc) : "memory");
  (void)m0;
}
__device__ inline void copy4(const v4i rsrc, uint32_t to, uint32_t from) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tbuffer_load_dword %2, %3, 0 offen lds" : "={m0}"(m0) : "s"(to), "v"(from), "s"(rsrc) : "memory");
  (void)m0;
}

// `most`: row tiles that groups in order can have; most * tiles_n fits 31 bits.
template <typename OUT, bool GATHER>
__global__ __launch_bounds__(64 * kWaves, 1) void grouped_wide_kernel(const Grouped a, int tiles_n, int most) {
  static_assert(sizeof(OUT) == 2, "rows of 64 outputs in 128 bytes");
  constexpr int TN = 4, kB = 4, kAll = 9;  // column tiles; a wave's copies of a stage: weights, rows and scales
  __shared__ __attribute__((aligned(1024))) int8_t lds[kLds];
  int* const before = reinterpret_cast<int*>(lds + kAtTiles);  // row tiles in front of each expert, [E + 1]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave / 4, wn = wave % 4;
  const int E = a.E, N = a.N, K = a.K;
  const int KB = (K + kBlock - 1) / kBlock, KB2 = (KB + 1) / 2 * 2;
  const int NB = (N + kBlock - 1) / kBlock;

  if (wave == 0) {
    int sum = 0;
    if (lane == 0) before[0] = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      int lo, hi;
      rows_of(a, e0 + lane, lo, hi);
      // descending offsets name rows more than once: no more tiles than rows in order make
      const int upto = min(sum + wave_inclusive(tiles_of_units((hi - lo + 63) / 64)), most);
      if (e0 + lane < E) before[e0 + lane + 1] = upto;
      sum = __builtin_amdgcn_readlane(upto, 63);
    }
  }
  __syncthreads();

  // This XCD's part of the list, and tile `turn` of this workgroup.
  const int total = __builtin_amdgcn_readfirstlane(before[E]) * tiles_n;
  const int xcd = (int)blockIdx.x % 8, slot = (int)blockIdx.x / 8;
  const int list = xcd * (total / 8) + min(xcd, total % 8), length = total / 8 + (xcd < total % 8 ? 1 : 0);
  const int step = (E + 63) / 64;
  auto tile_at = [&](int turn) __attribute__((always_inline)) {
    Tile t{0, 0, 0, 0, 4};
    int at = turn * kSlots + slot, half = -1;
    const int last = length - turn * kSlots;  // left for this turn
    if (last > 0 && 2 * last <= kSlots) {     // the last one: two workgroups a tile
      at = turn * kSlots + slot / 2;
      half = slot % 2;
    }
    if (at >= length) return t;
    const int id = list + at, mt = id / tiles_n;
    // the expert: 64 steps through the list, then one step
    uint64_t past = __ballot(before[min(E, (lane + 1) * step)] > mt);
    const int e0 = (int)__builtin_ctzll(past) * step;
    past = __ballot(lane < step && before[min(E, e0 + lane + 1)] > mt);
    t.expert = e0 + (int)__builtin_ctzll(past);
    const int front = uniform(before[t.expert]);
    const int lo = min(max(scalar(a.offsets, t.expert), 0), a.R), hi = min(max(scalar(a.offsets, t.expert + 1), lo), a.R);
    int tm, tn;
    const int units = (hi - lo + 63) / 64, tiles = tiles_of_units(units);
    tile_of(id - front * tiles_n, tiles, tiles_n, tm, tn);
    int u0 = begin_of(tm, tiles, units), u1 = begin_of(tm + 1, tiles, units);
    if (half >= 0) {
      const int cut = (u0 + u1 + 1) / 2;
      if (half == 0) u1 = cut;
      else u0 = cut;
    }
    t.m0 = lo + 64 * u0;
    t.rows = min(hi, lo + 64 * u1) - t.m0;
    t.n0 = tn * kColumns;
    t.height = 2 * max(u1 - u0, 2);
    return t;
  };

  // Copies.  Copy c of the rows is rows 64 c + 8 wave .. + 7 of the tile, of the
  // weights likewise.
  auto swz_a = [](int row) { return (row >> 1) & 7; };
  auto swz_b = [](int row) { return ((row >> 1) & 1) | (((row >> 4) & 3) << 1); };
  const uint32_t lx0 = tiled::dma::lds_addr(lds), lw0 = lx0 + kAtW, ls0 = lx0 + kAtScales, lr0 = lx0 + kAtRows;
  struct CopyPlace {
    int crow, srow;     // row of a copy, + 64 c; and whose scale this lane copies: every scale is copied twice
    uint32_t ca, cb, woff;
  };
  auto copy_place = [&]() __attribute__((always_inline)) {
    const int at = (int)fresh(threadIdx.x), crow = at >> 3;  // wave 8 + lane / 8
    return CopyPlace{crow, at & 255, (uint32_t)(((at & 7) ^ swz_a(crow)) * 16),
                     (uint32_t)(((at & 7) ^ swz_b(crow)) * 16),
                     (uint32_t)((crow & 7) * K + ((at & 7) ^ swz_b(crow)) * 16)};
  };
  CopyPlace cp = copy_place();
  struct Source {
    v4i ra, rb;
    const float* sa;
    int scales;             // bytes of sa that may be read
    const float* sw;
    uint32_t from[4], from_s;
  };
  Source src;
  if constexpr (GATHER) {
    src.ra = tiled::dma::rsrc_words(a.q, (int64_t)a.M * K);
    src.sa = a.s_a;
    src.scales = 0;
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) src.from[c] = (uint32_t)((64 * c + cp.crow) * K) + cp.ca;
    src.from_s = (uint32_t)cp.srow * 4u;
  }
  // Row numbers of tile t into buffer `buf` (zeros past its rows).
  auto copy_rows = [&](const Tile& t, int buf) __attribute__((always_inline)) {
    const v4i rr = tiled::dma::rsrc_words(a.rows + t.m0, (int64_t)t.rows * 4);
    copy4(rr, lr0 + (uint32_t)((buf * kRows + (wave & 3) * 64) * 4), (uint32_t)(fresh(threadIdx.x) & 255) * 4u);
  };
  // From here on the copies are of tile t (its row numbers are in buffer `buf`).
  auto copy_from = [&](const Tile& t, int buf) __attribute__((always_inline)) {
    src.rb = tiled::dma::rsrc_words(a.w + ((size_t)t.expert * (size_t)N + (size_t)t.n0) * (size_t)K,
                                    t.rows > 0 ? (int64_t)(N - t.n0) * K : 0);
    if constexpr (GATHER) {
      const int* numbers = reinterpret_cast<const int*>(lds + kAtRows) + buf * kRows;
      const CopyPlace cp = copy_place();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t m = (uint32_t)numbers[64 * c + cp.crow];
        src.from[c] = ((64 * c + cp.crow < t.rows) & (m < (uint32_t)a.M)) ? m * (uint32_t)K + cp.ca : kOutOfRange;
      }
      const uint32_t m = (uint32_t)numbers[cp.srow];
      src.from_s = ((cp.srow < t.rows) & (m < (uint32_t)a.M)) ? m * 4u : kOutOfRange;
      src.scales = a.M * 4;
    } else {
      src.ra = tiled::dma::rsrc_words(a.q + (size_t)t.m0 * (size_t)K, (int64_t)t.rows * K);
      src.sa = a.s_a + t.m0;
      src.scales = t.rows * 4;
    }
  };
  auto weight_scales = [&](const Tile& t) __attribute__((always_inline)) {
    const int nb = min((t.n0 + wn * 64) / kBlock, NB - 1);
    return a.s_w + ((size_t)t.expert * (size_t)NB + (size_t)nb) * (size_t)KB;
  };
  auto copy_x = [&](int c, int b, int buf) __attribute__((always_inline)) {
    const uint32_t ck = (uint32_t)b * kBlock;
    copy16(src.ra, lx0 + (uint32_t)(buf * kXBuf + (64 * c + wave * 8) * kBlock),
                            cp.ca + ck < (uint32_t)K ? src.from[c] + ck : kPast);
  };
  auto copy_w = [&](int c, int b, int buf) __attribute__((always_inline)) {
    const uint32_t ck = (uint32_t)b * kBlock;
    const int row = 64 * c + wave * 8;
    const uint32_t in = fresh(cp.woff) + ((uint32_t)(row * K) + ck);  // not in a branch: it would split the stage
    copy16(src.rb, lw0 + (uint32_t)(buf * kWBuf + row * kBlock),
                            cp.cb + ck < (uint32_t)K ? in : kPast);
  };
  auto copy_s = [&](int b, int buf) __attribute__((always_inline)) {
    const v4i rs = tiled::dma::rsrc_words(src.sa + (size_t)min(b, KB - 1) * (size_t)a.M, b < KB ? src.scales : 0);
    copy4(rs, ls0 + (uint32_t)((buf * kRows + (wave & 3) * 64) * 4), src.from_s);
  };

  // Where this lane reads: computed for each tile, since what is held over all of
  // them has no registers.
  struct Place {
    int xrow, xat, wat0;
  };
  auto place = [&]() __attribute__((always_inline)) {
    const int at = (int)fresh(threadIdx.x) & 63, r = at & 15, g = at >> 4;
    const int xrow = wm * 16 + r, wrow = wn * 64 + 16 * (r >> 2) + (r & 3);  // xrow + 32 i
    return Place{xrow, xrow * kBlock + ((g ^ swz_a(xrow)) * 16), wrow * kBlock + ((g ^ swz_b(wrow)) * 16)};
  };
  Place me = place();
  const float* const lsa = reinterpret_cast<const float*>(lds + kAtScales);
  auto read_x = [&](int buf, int i) __attribute__((always_inline)) {
    const int8_t* p = lds + buf * kXBuf + i * 32 * kBlock;
    return Frag16{*reinterpret_cast<const v4i*>(p + me.xat), *reinterpret_cast<const v4i*>(p + (me.xat ^ 64))};
  };
  auto read_w = [&](int buf, int j) __attribute__((always_inline)) {
    const int8_t* p = lds + kAtW + buf * kWBuf + j * 4 * kBlock;
    const int wat = (int)fresh((uint32_t)me.wat0);
    return Frag16{*reinterpret_cast<const v4i*>(p + wat), *reinterpret_cast<const v4i*>(p + (wat ^ 64))};
  };
  auto read_s = [&](int buf, int i) __attribute__((always_inline)) { return lsa[buf * kRows + me.xrow + 32 * i]; };

  Tile cur = tile_at(0), next;
  if (cur.rows <= 0) return;
  if constexpr (GATHER) {
    copy_rows(cur, 0);
    tiled::dma::wait_vmcnt<0>();
    barrier();
  }
  copy_from(cur, 0);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int c = 0; c < kB; ++c) copy_w(c, b, b);
    copy_x(0, b, b);
    copy_s(b, b);
#pragma unroll
    for (int c = 1; c < 4; ++c) copy_x(c, b, b);
  }
  const float* swp = weight_scales(cur);
  tiled::dma::wait_vmcnt<kAll>();
  barrier();
  float sw_next = scalar(swp, 0);

  // The stages and outputs of tile cur, and the copies of next's first two stages.
  // Nothing but scalars is held from tile to tile.
  auto body = [&](auto height, int buf_next, const float* swp_next) __attribute__((always_inline)) {
    constexpr int TM = decltype(height)::value;
    constexpr int QI = TM >= 6 ? 2 : 0, kPairsQ = (QI + 2) / 2;
    constexpr int nQ = kB + kPairsQ, nP = kAll - nQ;
    constexpr int kT = TN * TM, kP = TN * (TM - 2), kQ = TN * QI;
    constexpr int kPerP = (nP + 2 * TN - 1) / (2 * TN), kPerQ = (nQ + kP - kQ - 1) / (kP - kQ);
    constexpr int kLag = 3;
    auto tile = [](int t) { return t < kP ? t / TN : TM - 2 + (t - kP) % 2; };
    auto col = [](int t) { return t < kP ? t % TN : (t - kP) / 2; };
    me = place();
    cp = copy_place();
    copy_from(cur, 1 - buf_next);
    Frag16 x[2], w0[TN], w1[TN];
    float sa[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i] = read_x(0, i);
      sa[i] = read_s(0, i);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) w0[j] = read_w(0, j);
    v4f f[kT], p[kLag];
#pragma unroll
    for (int t = 0; t < kT; ++t) f[t] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < kLag; ++t) p[t] = v4f{0, 0, 0, 0};
    float scp[2] = {0.0f, 0.0f};
    auto fold = [&](int i, int j, const v4f& pv, float sc) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[TN * i + j][e] = __builtin_fmaf(pv[e], sc, f[TN * i + j][e]);
    };
    // Stage b in buffer buf; copies stage cbk of src behind it.
    auto stage = [&](int b, int cbk, const int buf, const float* sw_at, const Frag16* wf, Frag16* wnext)
                     __attribute__((always_inline)) {
      const float sw = fp8::uniform(b < KB ? sw_next : -0.0f);
      Operand16<false> wo[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) wo[j] = Operand16<false>(wf[j]);
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
        const v4f pn = block_sum(wo[j], Operand16<false>(xs[i]));
        __builtin_amdgcn_sched_barrier(0);
        if (t == kP || t == kQ) {
          wait_lgkm0();  // this wave's reads of what is handed back
          // the next stage's weights, rows 0 .. 127 and scales, its first seven
          // copies whichever height issued them; at Q, all of this stage's
          if (t == kP) tiled::dma::wait_vmcnt<kAll + nQ - 7>();
          else tiled::dma::wait_vmcnt<kAll>();
          barrier();
        }
        if (t < kP && j == 0) {
          xs[i + 2] = read_x(buf, i + 2);
          ss[i + 2] = read_s(buf, i + 2);
        }
        if (t == kP || t == kP + TN) {
          const int n = (t - kP) / TN;
          x[n] = read_x(1 - buf, n);
          sa[n] = read_s(1 - buf, n);
        }
        if (t >= kP && (t - kP) % 2 == 1) wnext[j] = read_w(1 - buf, j);
        if (t == kP + 1) sw_next = scalar(sw_at, 0);
        if (t >= kP) {
#pragma unroll
          for (int c = (t - kP) * kPerP; c < (t - kP + 1) * kPerP; ++c)
            if (c == 0) copy_s(cbk, buf);
            else if (c < nP) copy_x(c - 1 + kPairsQ, cbk, buf);
        } else if (t >= kQ) {
#pragma unroll
          for (int c = (t - kQ) * kPerQ; c < (t - kQ + 1) * kPerQ; ++c)
            if (c < kB) copy_w(c, cbk, buf);
            else if (c < nQ) copy_x(c - kB, cbk, buf);
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
    for (int b = 0; b < KB2 - 2; b += 2) {
      stage(b, b + 2, 0, swp + b + 1, w0, w1);
      stage(b + 1, b + 3, 1, swp + b + 2, w1, w0);
    }
    copy_from(next, buf_next);
    stage(KB2 - 2, 0, 0, swp + KB - 1, w0, w1);
    stage(KB2 - 1, 1, 1, swp_next, w1, w0);
#pragma unroll
    for (int t = 0; t < kLag; ++t) fold(tile(kT - kLag + t), col(kT - kLag + t), p[t], scp[(kT - kLag + t) % 2]);

    // The sums are done here: the compiler would move the last two stages' into the
    // branches that store them, and hold the products until then.
#pragma unroll
    for (int t = 0; t < kT; ++t) asm volatile("" : "+v"(f[t]));

    // A lane holds 16 consecutive columns of one of 16 rows: through LDS (the wave's own
    // part, beside the stages) they are stored as whole rows.
    const int at = (int)fresh(threadIdx.x) & 63, ra = at & 15, ga = at >> 4;  // computed here, not held over the stages
    int8_t* const part = lds + kAtOut + wave * 16 * kPitch;
    const int n = cur.n0 + wn * 64 + at % 8 * 8;
    OUT* const y = static_cast<OUT*>(a.y) + (size_t)cur.m0 * (size_t)N;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int c = 0; c < 16; c += 8) {
        OUT o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rounded<OUT>(f[TN * i + (c + e) / 4][e % 4]);
        __builtin_memcpy(__builtin_assume_aligned(part + ra * kPitch + (16 * ga + c) * 2, 16), o, 16);
      }
      wave_order();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = at / 8 + t * 8, m = 32 * i + 16 * wm + row;
        OUT o[8];
        __builtin_memcpy(o, __builtin_assume_aligned(part + row * kPitch + at % 8 * 16, 16), 16);
        if (m >= cur.rows) continue;
        OUT* yr = y + (size_t)m * (size_t)N;
        if (n + 8 <= N) {
          __builtin_memcpy(yr + n, o, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) yr[n + e] = o[e];
        }
      }
      wave_order();
    }
  };
  for (int turn = 1;; ++turn) {
    next = tile_at(turn);
    if (next.rows < 0) next.rows = 0;
    if constexpr (GATHER) copy_rows(next, turn & 1);
    const float* const swp_next = weight_scales(next);
    if (cur.height == 8) body(std::integral_constant<int, 8>{}, turn & 1, swp_next);
    else if (cur.height == 6) body(std::integral_constant<int, 6>{}, turn & 1, swp_next);
    else body(std::integral_constant<int, 4>{}, turn & 1, swp_next);
    if (next.rows <= 0) break;
    cur = next;
    swp = swp_next;
  }
  tiled::dma::wait_vmcnt<0>();  // the copies behind the last tile have landed
}

}  // namespace wide
}  // namespace fp8
}  // namespace prism
