// fp8 (e4m3) GEMM grouped by expert, with ragged groups: rows offsets[e] ..
// offsets[e + 1] - 1 of the output come from expert e's weights.  The arithmetic
// is that of gemm_fp8.hip on the same instructions, so that a row has the bits that
// the dense product with its expert's weights gives it: for a bf16 y those of the fp8
// instruction, which cuts small products beside large ones, as explained there.
//
// The groups are known on the device only: the grid is the largest number of row
// tiles that the sizes allow, each workgroup finds its tile from the offsets, and
// those past the last one leave at once.
//
// Groups of few rows are bound by reading their experts' weights: 17 x 8 rows of 128
// groups, 2560 x 4096 bf16, 110 us (625 MB and more: 5.7 TB/s); 1 x 8 of 64, 2560 x 2560,
// 11.5 (52 MB, 4.6 TB/s).  Between them and the wide tiles, which are bound as the
// dense product's are, short tiles whose rows are in part empty: 611 x 4 of 60, 2576 x
// 1472 fp16, 69 us (48 for the bytes; VALU 58% active, MFMA 27% busy).
#include "gemm_fp8_grouped_wide.h"

namespace prism {
namespace {

using namespace fp8;

// Tiles of BM rows that expert e's rows lo .. hi - 1 make.
template <int BM>
__device__ inline int tiles_of(const Grouped& a, int e, int& lo, int& hi) {
  rows_of(a, e, lo, hi);
  return (hi - lo + BM - 1) / BM;
}

struct Group {
  int expert, begin, end;  // rows begin .. end - 1 of y
  int tile, tiles;         // the row tile found, of how many
};

// The group that has row tile `id` of all groups' tiles of BM rows; false past the last.
template <int BM>
__device__ inline bool find_group(const Grouped& a, int id, Group& g) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    int lo, hi;
    const int tiles = tiles_of<BM>(a, e0 + lane, lo, hi);
    const int upto = wave_inclusive(tiles);
    const uint64_t reach = __ballot(upto > id);
    if (reach) {
      const int at = (int)__builtin_ctzll(reach);
      g.expert = e0 + at;
      g.begin = __builtin_amdgcn_readlane(lo, at);
      g.end = __builtin_amdgcn_readlane(hi, at);
      g.tiles = __builtin_amdgcn_readlane(tiles, at);
      g.tile = id - (__builtin_amdgcn_readlane(upto, at) - g.tiles);
      return true;
    }
    id -= __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// Row tiles of all groups.
template <int BM>
__device__ inline int count_tiles(const Grouped& a) {
  int n = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    int lo, hi;
    n += __builtin_amdgcn_readlane(wave_inclusive(tiles_of<BM>(a, e0 + (threadIdx.x & 63), lo, hi)), 63);
  }
  return n;
}

// Few rows, fp32 and f16 y: as the dense product's kernel for few rows, bound by reading
// the weights once.  A workgroup owns 16 rows of a group and 16 columns, and its waves
// share out K: in rounds of kWaves blocks, each wave multiplies its block straight from
// global memory and leaves the sums in LDS with the blocks' scales; after one
// barrier, threads fold the round's blocks into their outputs in order.  A bf16 y,
// whose operands need no conversion, never takes this kernel.
constexpr int kWaves = 4;
template <typename OUT>
__global__ __launch_bounds__(64 * kWaves) void grouped_small_kernel(const Grouped a, int tiles_n) {
  constexpr int kTile = 16 * 16;
  static_assert(kTile == 64 * kWaves, "one output a thread");
  __shared__ __attribute__((aligned(16))) float lp[2][kWaves][kTile];
  __shared__ float ls[2][kWaves][16];
  Group t;
  if (!find_group<16>(a, (int)(blockIdx.x / (unsigned)tiles_n), t)) return;
  const int first = t.begin + t.tile * 16, rows = min(16, t.end - first);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int N = a.N, K = a.K;
  const int n0 = (int)(blockIdx.x % (unsigned)tiles_n) * 16;
  const int KB = (K + kBlock - 1) / kBlock, NB = (N + kBlock - 1) / kBlock;
  const uint8_t* w = a.w + ((size_t)t.expert * (size_t)N + (size_t)n0) * (size_t)K;
  const auto rw = make_rsrc(w, (int64_t)(N - n0) * K);
  const float* swp = a.s_w + ((size_t)t.expert * (size_t)NB + (size_t)(n0 / kBlock)) * (size_t)KB;

  // q's row of this lane's row: -1 past the tile or outside q
  int m = -1;
  if (r < rows) m = a.rows ? a.rows[first + r] : first + r;
  if ((uint32_t)m >= (uint32_t)a.M) m = -1;
  const uint8_t* const xp = a.q + (size_t)max(m, 0) * (size_t)K;

  struct Round {
    Frag16 x, w;
    float sa, sw;
  };
  auto load = [&](int b0, Round& d) __attribute__((always_inline)) {
    const int b = b0 + wave;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = b * kBlock + 16 * g + 64 * h;
      const bool in = k < K;
      d.x.c[h] = in && m >= 0 ? *reinterpret_cast<const v4i*>(xp + k) : v4i{0, 0, 0, 0};
      d.w.c[h] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? (uint32_t)(r * K + k) : kOutOfRange, 0, 0);
    }
    const int bb = b < KB ? b : KB - 1;  // blocks past K are not folded
    d.sa = m < 0 ? 0.0f : a.s_a[(size_t)bb * (size_t)a.M + (size_t)m];
    d.sw = swp[bb];
  };
  auto multiply = [&](int buf, const Round& d) __attribute__((always_inline)) {
    *reinterpret_cast<v4f*>(&lp[buf][wave][(g * 16 + r) * 4]) = block_sum(Operand16<true>(d.w), Operand16<true>(d.x));
    if (lane < 16) ls[buf][wave][lane] = d.sa * d.sw;
  };
  // thread e: column 4 (e / 64) + e % 4 of row e / 4 % 16
  const int e = (int)threadIdx.x, row = e / 4 % 16;
  float f = 0.0f;
  Round cur, next;
  load(0, cur);
  int buf = 0;
  for (int b0 = 0; b0 < KB; b0 += kWaves) {
    load(b0 + kWaves, next);
    multiply(buf, cur);
    __syncthreads();  // also: every thread is done folding the round before last out of the other buffer
    const int count = KB - b0 < kWaves ? KB - b0 : kWaves;
    for (int b = 0; b < count; ++b) f = __builtin_fmaf(lp[buf][b][e], ls[buf][b][row], f);
    cur = next;
    buf ^= 1;
  }
  const int n = n0 + 4 * (e / 64) + e % 4;
  if (row < rows && n < N) static_cast<OUT*>(a.y)[(size_t)(first + row) * (size_t)N + (size_t)n] = rounded<OUT>(f);
}

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of BM rows that the groups can have at the most: each group's last
// one may be short, and none is empty.
int64_t most_tiles(int64_t R, int64_t E, int64_t BM) {
  const int64_t groups = R < E ? R : E;
  return (R + groups * (BM - 1)) / BM;
}

int check_grid(int64_t groups, int threads) {
  return groups * threads <= (int64_t)UINT32_MAX ? PRISM_OK : PRISM_ERR_INVALID_ARG;
}

template <typename OUT>
int launch_small(const Grouped& a, hipStream_t st, bool check) {
  const int64_t tiles_n = ceil_div(a.N, 16), groups = tiles_n * most_tiles(a.R, a.E, 16);
  if (check) return check_grid(groups, 64 * kWaves);
  grouped_small_kernel<OUT><<<(unsigned)groups, 64 * kWaves, 0, st>>>(a, (int)tiles_n);
  return launch_status();
}

// Many rows a group: the dense product's LDS tiles, 32 TM rows by 16 TN WN columns,
// ordered expert by expert; a group's last tile is one of 32 TAIL rows where that is
// enough.
template <typename OUT, bool EXACT, int WN, int TM, int TN, int R, int TAIL, int OCC, bool GATHER>
__global__ __launch_bounds__(128 * WN, OCC) void grouped_tile_kernel(const Grouped a, int tiles_n) {
  constexpr int kLds = kTileLds<WN, TM, TN, R>;
  static_assert(TAIL <= TM && kLds <= 160 * 1024 / OCC, "LDS");
  __shared__ __attribute__((aligned(1024))) int8_t lds[kLds];
  const int total = count_tiles<32 * TM>(a) * tiles_n;
  if ((int)blockIdx.x >= total) return;
  const int id = xcd_order((int)blockIdx.x, total);
  Group t;
  if (!find_group<32 * TM>(a, id / tiles_n, t)) return;
  int tm, tn;
  tile_of(t.tile * tiles_n + id % tiles_n, t.tiles, tiles_n, tm, tn);
  const int N = a.N, K = a.K;
  const int m0 = t.begin + tm * 32 * TM, n0 = tn * 16 * TN * WN;
  const uint8_t* w = a.w + (size_t)t.expert * (size_t)N * (size_t)K;
  const float* s_w = a.s_w + (size_t)t.expert * (size_t)ceil_div(N, kBlock) * (size_t)ceil_div(K, kBlock);
  if (TAIL == TM || t.end - m0 > 32 * TAIL)
    tile_body<OUT, EXACT, WN, TM, TN, R, false, GATHER>(lds, a.q, a.s_a, a.M, w, s_w, static_cast<OUT*>(a.y), t.end, N,
                                                        K, m0, n0, {a.rows, a.M});
  else if constexpr (TAIL < TM)
    tile_body<OUT, EXACT, WN, TAIL, TN, R, false, GATHER>(lds, a.q, a.s_a, a.M, w, s_w, static_cast<OUT*>(a.y), t.end,
                                                          N, K, m0, n0, {a.rows, a.M});
}

template <typename OUT, bool EXACT, int WN, int TM, int TN, int R, int TAIL, int OCC>
int launch_tile(const Grouped& a, hipStream_t st, bool check) {
  const int64_t tiles_n = ceil_div(a.N, 16 * TN * WN), groups = tiles_n * most_tiles(a.R, a.E, 32 * TM);
  if (check) return check_grid(groups, 128 * WN);
  if (a.rows)
    grouped_tile_kernel<OUT, EXACT, WN, TM, TN, R, TAIL, OCC, true><<<(unsigned)groups, 128 * WN, 0, st>>>(a, (int)tiles_n);
  else
    grouped_tile_kernel<OUT, EXACT, WN, TM, TN, R, TAIL, OCC, false><<<(unsigned)groups, 128 * WN, 0, st>>>(a, (int)tiles_n);
  return launch_status();
}

template <typename OUT>
int launch_wide(const Grouped& a, hipStream_t st, bool check) {
  // rows are counted in whole tiles, in 32 bits
  if (check) return a.R <= INT32_MAX - wide::kRows ? PRISM_OK : PRISM_ERR_INVALID_ARG;
  const int tiles_n = (int)ceil_div(a.N, wide::kColumns), most = (int)most_tiles(a.R, a.E, wide::kRows);
  constexpr unsigned kGroups = 8 * wide::kSlots;
  if (a.rows)
    wide::grouped_wide_kernel<OUT, true><<<kGroups, 64 * wide::kWaves, 0, st>>>(a, tiles_n, most);
  else
    wide::grouped_wide_kernel<OUT, false><<<kGroups, 64 * wide::kWaves, 0, st>>>(a, tiles_n, most);
  return launch_status();
}

// Kernel for (R, E, N), fitted on MI355X with weights from HBM (us below) at K = 2560 alone:
// other K are taken to stretch all forms alike, which was not measured.  Groups are not
// known here: as many as can have rows are taken to, each with half a tile more than
// its rows fill.  Estimates count rounds of the tiles that run at once:
//  * an fp32 or f16 y: the kernel for few rows while its workgroups are few (8
//    groups of 6 rows by 2560 columns: 14.7, 64 x 64 tiles 18.3; of 16 rows 22.4 and
//    18.9), else 64 x 64 or 128 x 128 tiles (64 groups by 640 columns: 48 rows 35 and
//    42, 96 rows 52 and 45, 512 rows 179 and 132);
//  * bf16: 64 x 64 tiles, 64 x 128 tiles, 128 x 128 tiles or the wide kernel (64
//    groups by 640: 6 rows 24.9, 26.3, 26.3 and 28.9; 64 rows 32.7, 28.9, 33.7 and 37.1;
//    128 rows 47.6, 44.3, 36.7 and 39.8; 512 rows 138, 114, 94 and 81.  By 2560: 6 rows
//    82, 80, 88 and 90; 512 rows 526, 443, 340 and 274).
template <bool EXACT>
int form_of(const Grouped& a) {
  const float R = (float)a.R, G = (float)(a.R < a.E ? a.R : a.E);
  auto tiles = [&](int bm, int bn) {
    const float in_column = R / (float)bm + 0.5f * G;
    return (in_column > G ? in_column : G) * (float)ceil_div(a.N, bn);
  };
  const float r64 = tiles(64, 64) / 768.0f, r128 = tiles(128, 128) / 512.0f;
  if constexpr (EXACT) {
    const float few = tiles(16, 16);
    if (few <= 720.0f || (few <= 1280.0f && R <= 8.0f * G)) return PRISM_GROUPED_FEW;
    const float c128 = r128 <= 0.5f ? 29.0f : r128 <= 1.0f ? 44.0f : 14.0f + 42.0f * r128;
    return 6.0f + 24.0f * r64 < c128 ? PRISM_GROUPED_64x64 : PRISM_GROUPED_128x128;
  } else {
    const float r64w = tiles(64, 128) / 512.0f, turns = tiles(wide::kRows, wide::kColumns) / 256.0f;
    const float c64 = r64 <= 0.33f ? 22.0f : r64 <= 0.87f ? 25.0f : 9.0f + 18.3f * r64;
    const float c64w = r64w <= 0.5f ? 24.0f : r64w <= 0.95f ? 27.0f : 9.0f + 19.0f * r64w;
    const float c128 = r128 <= 1.0f ? 35.0f : r128 <= 2.0f ? 60.0f : 10.0f + 29.0f * r128;
    const bool can = a.K >= wide::kMinK && most_tiles(a.R, a.E, wide::kRows) * ceil_div(a.N, wide::kColumns) <= INT32_MAX;
    const float cwide = can ? 20.5f * (float)(int64_t)(2.0f * (turns > 1.0f ? turns : 1.0f) + 0.99f) : 3e38f;
    const float best = fminf(fminf(c64, c64w), fminf(c128, cwide));
    return best == c64 ? PRISM_GROUPED_64x64 : best == c64w ? PRISM_GROUPED_64x128
                                             : best == c128 ? PRISM_GROUPED_128x128 : PRISM_GROUPED_WIDE;
  }
}

template <typename OUT, bool EXACT>
int launch(const Grouped& a, hipStream_t st, bool check) {
  const int form = form_of<EXACT>(a);
  if (form == PRISM_GROUPED_64x64) return launch_tile<OUT, EXACT, 2, 2, 2, 3, 2, 3>(a, st, check);
  if (form == PRISM_GROUPED_128x128) return launch_tile<OUT, EXACT, 2, 4, 4, 2, 2, 2>(a, st, check);
  if constexpr (EXACT) {
    return launch_small<OUT>(a, st, check);
  } else {
    if (form == PRISM_GROUPED_64x128) return launch_tile<OUT, EXACT, 4, 2, 2, 3, 2, 2>(a, st, check);
    return launch_wide<OUT>(a, st, check);
  }
}

int dispatch(const Grouped& a, int type, hipStream_t st, bool check) {
  if (type == PRISM_TYPE_F32) return launch<float, true>(a, st, check);
  if (type == PRISM_TYPE_F16) return launch<_Float16, true>(a, st, check);
  return launch<__bf16, false>(a, st, check);
}

}  // namespace

int check_gemm_fp8_grouped_grid(int type, int R, int E, int N, int K) {
  return dispatch({nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, R, E, N, K}, type, nullptr, true);
}

int gemm_fp8_grouped_form(int type, int R, int E, int N, int K) {
  const Grouped a{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, R, E, N, K};
  return type == PRISM_TYPE_BF16 ? form_of<false>(a) : form_of<true>(a);
}

int launch_gemm_fp8_grouped(const uint8_t* q, const float* s_a, const int32_t* rows, const int32_t* offsets,
                            const uint8_t* w, const float* s_w, void* y, int type, int M, int R, int E, int N, int K,
                            hipStream_t st) {
  return dispatch({q, s_a, rows, offsets, w, s_w, y, M, R, E, N, K}, type, st, false);
}

}  // namespace prism
