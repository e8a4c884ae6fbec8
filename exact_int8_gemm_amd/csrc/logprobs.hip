// Token read-out: log probabilities of given tokens, the entropy and the top
// alternatives of each row of logits (the method's engine answers typed
// questions from the probabilities of given tokens after one forward pass;
// StartLux-Prism README, "Example" and "How it works").
//
// With m = max z, S = sum exp(z - m), W = sum exp(z - m) (z - m):
//   lse = m + log S, logprob(t) = (z_t - m) - log S, entropy = log S - W / S.
// Both terms of the entropy are >= 0, so nothing cancels.  m, S and W are
// fp32; exp is one v_exp_f32 of (z - m) log2(e), whose error (|z - m| 2^-24
// relative) is largest where the term itself vanishes.
//
// The vocabulary axis is cut into chunks of kChunk values whatever M is, one
// wave each, so a row's sums are always added in the same order.  A chunk is
// read once and stays in registers: maximum, sums, and its `top` largest
// values; a second kernel joins the chunks of a row.  Waves do not wait for
// each other.  2048 x 100003 bf16, both kernels, calls back to back from HBM: 96
// us with top 8, 75 without (410 MB: 81 us at a large copy's rate; traced one
// launch at a time 103 and 8.6).  With four waves and five barriers to
// each 8192 values, which left the vector units idle 40% of the time, it took
// 150 us.  What bounds it now is issue: per value an exp at a quarter of the
// rate and six other instructions; held to 96 or fewer registers for more
// waves, the kernel spills (105 us).
//
// Top values: a bisection finds a value t that at least `top` of the 64 lanes'
// maxima reach, and often no more.  Only the 16-byte pieces with values of at
// least t are looked at, through LDS (95 us; all values of the lanes that have
// such, 102; of all lanes, 144); those values, a few more than `top`, are
// ranked by value and then by index, as one 64-bit key each.  When too many
// values tie at t (a chunk masked to one finite value), the larger ones are
// ranked and the tied ones marked, of which the first are taken; the join then
// merges the chunks' sorted keys (256 x 100003 f16, all of the lowest value, top
// 20: 29 us, about what random values take; 51 MB).  The slowest rows are those whose
// large values, more than are ranked at once, share few lanes: their lanes are
// visited once for each listed value (256 x 100003 bf16, top 32: random 30 us,
// ascending 471, large ones in 4 to 31 lanes 431 to 449; fp32 ascending 37, large
// ones in 4 lanes 411).
#include "../../include/prism.h"
#include "prism_internal.h"
#include "wave.h"

namespace prism {
namespace {

constexpr int kPerLane = 64;
constexpr int kChunk = 64 * kPerLane;
constexpr int kCand = 128;  // candidates of a chunk ranked at once
constexpr int kPieces = 64; // 16-byte pieces with candidates that are held in LDS
constexpr int kHold = 16;   // lanes whose values are held there at once
constexpr int kJoinCand = 1024;
constexpr int kRankCand = 128;  // of the keys of up to 64 chunks: more are merged
constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2E = 0x1.715476p+0f, kLn2 = 0x1.62e430p-1f;
constexpr float kNegInf = -__builtin_inff();
// Lowest exponent of 2 taken: 2^-200 is 0 in fp32, and unlike -inf it can be
// multiplied by that.
constexpr float kFloor = -200.0f;
// Largest |m| of a chunk whose terms take one fma each: the rounding of m
// log2(e), by which all their exponents are off, is at most 2^-4.
constexpr float kOneFma = 0x1p20f;

struct Stats {
  float m, S, W;
};

// Keys order values first, then lower indices; 0 is below every key of a
// value above -inf.  + 0.0f makes -0 equal to 0.
__device__ inline uint32_t order_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ inline float of_order(uint32_t o) {
  return __builtin_bit_cast(float, (o >> 31) ? (o & 0x7fffffffu) : ~o);
}
__device__ inline uint64_t key_of(float v, uint32_t index) {
  return ((uint64_t)order_of(v) << 32) | (uint32_t)~index;
}
__device__ inline float value_of(uint64_t key) { return of_order((uint32_t)(key >> 32)); }
__device__ inline uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

template <typename T>
__device__ inline float to_float(T v) {
  return (float)v;
}

// Value e of 16 bytes of values, as fp32; the last argument names their type.
__device__ inline float value_at(const v4i p, int e, const float*) {
  return __builtin_bit_cast(float, (uint32_t)p[e]);
}
__device__ inline float value_at(const v4i p, int e, const __bf16*) {
  const uint32_t w = (uint32_t)p[e / 2];
  return __builtin_bit_cast(float, e % 2 ? w & 0xffff0000u : w << 16);
}
__device__ inline float value_at(const v4i p, int e, const _Float16*) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)((uint32_t)p[e / 2] >> (e % 2 * 16)));
}

// m = -inf (nothing in the row or chunk) as the base of z - m.
__device__ inline float base_of(float m) { return m == kNegInf ? 0.0f : m; }

// log2 of the term exp(d), floored; a NaN stays one.
__device__ inline float log2_term(float d) { return __builtin_elementwise_maximum(d * kLog2E, kFloor); }

__device__ inline uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ inline uint64_t shfl_xor_u64(uint64_t v, int off) {
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, off, 64);
  const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), off, 64);
  return ((uint64_t)hi << 32) | lo;
}

// Reductions over a wave without LDS (data-parallel primitives: shifts within
// rows of 16 lanes, then row broadcasts), the result in every lane.
template <int CTRL, int ROWS>
__device__ inline float dpp(float v, float old) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                                               CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false));
}
__device__ inline uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xf>(v);  // the steps of wave_reduce below
  v = dpp_max<0x112, 0xf>(v);
  v = dpp_max<0x114, 0xf>(v);
  v = dpp_max<0x118, 0xf>(v);
  v = dpp_max<0x142, 0xa>(v);
  v = dpp_max<0x143, 0xc>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline uint64_t wave_max_key(uint64_t k) {
  const uint32_t hi = wave_max((uint32_t)(k >> 32));
  const uint32_t lo = wave_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}
template <typename F>
__device__ inline float wave_reduce(float v, float neutral, F op) {
  v = op(v, dpp<0x111, 0xf>(v, neutral));  // row_shr:1
  v = op(v, dpp<0x112, 0xf>(v, neutral));  // row_shr:2
  v = op(v, dpp<0x114, 0xf>(v, neutral));  // row_shr:4
  v = op(v, dpp<0x118, 0xf>(v, neutral));  // row_shr:8
  v = op(v, dpp<0x142, 0xa>(v, neutral));  // row_bcast:15 into rows 1 and 3
  v = op(v, dpp<0x143, 0xc>(v, neutral));  // row_bcast:31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ inline float wave_max(float v) {
  return wave_reduce(v, kNegInf, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
}
__device__ inline float wave_min(float v) {
  return wave_reduce(v, -kNegInf, [](float a, float b) { return fminf(a, b); });
}
__device__ inline float wave_sum(float v) {
  return wave_reduce(v, 0.0f, [](float a, float b) { return a + b; });
}

// A value that at least `top` (<= 64) of the lanes' values reach, and often no
// more of them: halvings of the ordered bit patterns between the values'
// minimum and maximum.
__device__ inline float kth_of_wave(float g, float largest, int top) {
  const uint32_t o = order_of(g);
  uint32_t lo = order_of(wave_min(g)), hi = order_of(largest) + 1;
  for (int i = 0; i < 16 && hi - lo > 1; ++i) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int n = __popcll(__ballot(o >= mid));
    if (n >= top) lo = mid;
    else hi = mid;
    if (n == top) break;
  }
  return of_order(__builtin_amdgcn_readfirstlane(lo));
}

// Lanes below this one in a mask.
__device__ inline int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

template <int NT>
__device__ inline uint64_t block_max_key(uint64_t v, uint64_t* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max_u64(v, shfl_xor_u64(v, off));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s = max_u64(s, lds[i]);
  __syncthreads();
  return s;
}

// The n distinct keys in LDS: those of rank < top go to out[rank].
template <int NT>
__device__ inline void rank_keys(const uint64_t* keys, int n, int top, uint64_t* out) {
  for (int i = threadIdx.x % NT; i < n; i += NT) {
    const uint64_t k = keys[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += keys[j] > k ? 1 : 0;
    if (rank < top) out[rank] = k;
  }
}

// Row results from the joined statistics and the sorted keys (0 = none) in
// LDS.
template <typename T, int NT>
__device__ inline void write_row(const T* z, int64_t V, int64_t row, const Stats st, const uint64_t* keys,
                                 const int64_t* tokens, int64_t ntok, int top, float* lp, float* lse, float* ent,
                                 int64_t* top_ids, float* top_lp) {
  const bool bad = st.S != st.S || st.m == -kNegInf;  // a NaN or +inf in the row
  const bool empty = !bad && st.m == kNegInf;
  const float base = base_of(st.m);
  const float ls = logf(st.S);
  const float nan = __builtin_nanf("");
  const int tid = (int)(threadIdx.x % NT);
  if (tid == 0) {
    if (lse) lse[row] = bad ? nan : empty ? kNegInf : base + ls;
    if (ent) ent[row] = bad ? nan : empty ? 0.0f : ls - st.W * kLn2 / st.S;
  }
  for (int64_t i = tid; i < ntok; i += NT) {
    const int64_t t = tokens[row * ntok + i];
    float r = nan;
    if (t >= 0 && t < V && !bad) r = empty ? kNegInf : (to_float(z[t]) - base) - ls;
    lp[row * ntok + i] = r;
  }
  for (int i = tid; i < top; i += NT) {
    const uint64_t k = keys[i];
    float r = kNegInf;
    if (k != 0 && !empty && !bad) r = (value_of(k) - base) - ls;
    top_lp[row * top + i] = bad ? nan : r;
    top_ids[row * top + i] = (bad || r == kNegInf) ? -1 : (int64_t)index_of(k);
  }
}

// Chunk u % chunks of row u / chunks, u = this wave: statistics and sorted top
// keys into stats[u] and keys[u][top]; or, if a row is one chunk, the row's
// results.
template <typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void logprobs_chunk_kernel(
    const T* __restrict__ logits, int64_t ld, int64_t V, unsigned total, int chunks, int top,
    Stats* __restrict__ stats, uint64_t* __restrict__ keys, const int64_t* __restrict__ tokens, int64_t ntok,
    float* __restrict__ lp, float* __restrict__ lse, float* __restrict__ ent, int64_t* __restrict__ top_ids,
    float* __restrict__ top_lp) {
  constexpr int kVec = 16 / (int)sizeof(T);
  constexpr int kIter = kPerLane / kVec;
  constexpr int kRow = kPerLane * (int)sizeof(T) + 16;  // 16 more bytes against bank conflicts
  __shared__ __attribute__((aligned(16))) uint8_t lheld[WAVES][kHold * kRow];
  static_assert(kHold * kRow >= kPieces * 16, "pieces share the lanes' LDS");
  __shared__ uint16_t lplaces[WAVES][kPieces];
  __shared__ uint64_t lcand[WAVES][kCand];
  __shared__ uint64_t lbest[WAVES][PRISM_TOP_MAX];
  __shared__ uint8_t ltied[WAVES][64 * kIter];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const unsigned u = blockIdx.x * WAVES + (unsigned)wave;
  if (u >= total) return;  // no barrier below
  uint8_t* held = lheld[wave];
  uint16_t* places = lplaces[wave];
  uint64_t* cand = lcand[wave];
  uint64_t* best = lbest[wave];
  uint8_t* tied = ltied[wave];
  const int64_t row = u / (unsigned)chunks;
  const int64_t base = (int64_t)(u % (unsigned)chunks) * kChunk;
  const T* z = logits + row * ld + base;

  // Value i of this lane is value place(i) of the chunk: pieces of kVec
  // consecutive ones.  A row may start at any element, so the 16-byte loads
  // are unaligned ones.  They stay as loaded and are converted at each use.
  auto place = [&](int i) { return ((i / kVec) * 64 + lane) * kVec + i % kVec; };
  v4i raw[kIter];
  if (V - base >= kChunk) {
#pragma unroll
    for (int it = 0; it < kIter; ++it) __builtin_memcpy(&raw[it], z + place(it * kVec), 16);
  } else {
    // the row's last chunk: -inf behind its end
    const int left = (int)(V - base);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const int at = place(it * kVec);
      T t[kVec];
      if (at + kVec <= left) {
        __builtin_memcpy(t, z + at, 16);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) t[e] = at + e < left ? z[at + e] : (T)kNegInf;
      }
      __builtin_memcpy(&raw[it], t, 16);
    }
  }
  auto value = [&](int i) __attribute__((always_inline)) { return value_at(raw[i / kVec], i % kVec, (const T*)nullptr); };
  float gm[kIter], mt = kNegInf;  // maxima of the pieces, and of all; a NaN stays one
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    gm[it] = value(it * kVec);
#pragma unroll
    for (int e = 1; e < kVec; ++e) gm[it] = __builtin_elementwise_maximum(gm[it], value(it * kVec + e));
    mt = __builtin_elementwise_maximum(mt, gm[it]);
  }
  Stats st;
  st.m = wave_max(mt);
  const float b = base_of(st.m);
  float S = 0.0f, W = 0.0f;  // W in powers of 2
  if (fabsf(b) < kOneFma) {
    // (v - b) log2(e) as one fma: v L - c with c = fl(b L).  Every term is then
    // 2^d too large for d = b L - c, which an fma gives exactly: taken out of
    // the sums below.  |d| is up to half a step of c, 2^-4 here; without a bound
    // on b, 2^d leaves fp32 from |b| = 1.5e9 on.
    const float c = b * kLog2E, d = __builtin_fmaf(b, kLog2E, -c);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const float t = __builtin_elementwise_maximum(__builtin_fmaf(value(i), kLog2E, -c), kFloor);
      const float e = __builtin_amdgcn_exp2f(t);
      S += e;
      W = __builtin_fmaf(e, t, W);
    }
    const float x = __builtin_amdgcn_exp2f(-d);
    S *= x;
    W = __builtin_fmaf(W, x, -d * S);
  } else {  // chunks masked to one finite value, mostly (a NaN also comes here)
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const float t = log2_term(value(i) - b);
      const float e = __builtin_amdgcn_exp2f(t);
      S += e;
      W = __builtin_fmaf(e, t, W);
    }
  }
  st.S = wave_sum(S);
  st.W = wave_sum(W);

  if (top > 0) {
    const float t = fmaxf(kth_of_wave(mt, st.m, top), kLowest);  // -inf is never listed
    if (lane < top) best[lane] = 0;
    int n = 0;
    auto collect = [&](bool in, float v, int at) __attribute__((always_inline)) {
      const uint64_t who = __ballot(in);
      const int to = n + lanes_below(who);
      if (in && to < kCand) cand[to] = key_of(v, (uint32_t)(base + at));
      n += __popcll(who);
    };
    // Pieces whose maximum is wanted go to LDS, to have a lane for each of their
    // values; where there are more than kPieces of them, only their number counts.
    auto gather = [&](auto&& wanted) __attribute__((always_inline)) {
      int np = 0;
      wave_order();
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const bool in = wanted(gm[it]);
        const uint64_t who = __ballot(in);
        if (!who) continue;
        const int to = np + lanes_below(who);
        if (in && to < kPieces) {
          *reinterpret_cast<v4i*>(held + to * 16) = raw[it];
          places[to] = (uint16_t)place(it * kVec);
        }
        np += __popcll(who);
      }
      wave_order();
      return np;
    };
    auto collect_pieces = [&](int np, auto&& wanted) __attribute__((always_inline)) {
      for (int i = lane; i - lane < np * kVec; i += 64) {
        const float v = to_float(reinterpret_cast<const T*>(held)[i]);  // of 64 kVec: past np stale ones
        collect(i < np * kVec && wanted(v), v, places[i / kVec] + i % kVec);
      }
    };
    // The lanes with values of at least t whole, one after the other; f returns
    // whether to go on.
    auto visit = [&](auto&& f) __attribute__((always_inline)) {
      wave_order();
      for (uint64_t left = __ballot(mt >= t); left != 0;) {
        const int slot = lanes_below(left);
        if ((left >> lane & 1) && slot < kHold) {
#pragma unroll
          for (int it = 0; it < kIter; ++it) *reinterpret_cast<v4i*>(held + slot * kRow + it * 16) = raw[it];
        }
        wave_order();
        for (int j = 0; j < kHold && left != 0; ++j, left &= left - 1) {
          const int src = __builtin_ctzll(left);
          const float v = to_float(reinterpret_cast<const T*>(held + j * kRow)[lane]);
          if (!f(v, ((lane / kVec) * 64 + src) * kVec + lane % kVec)) return;
        }
        wave_order();
      }
    };
    auto reaches = [&](float v) { return v >= t; };
    auto exceeds = [&](float v) { return v > t; };
    int np = gather(reaches);
    if (np <= kPieces) collect_pieces(np, reaches);
    if (np > kPieces || n > kCand) {
      // Many values tie at t: rank the larger ones, mark the tied ones, a byte
      // for each piece.
      n = 0;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) m |= value(it * kVec + e) == t ? 1u << e : 0u;
        tied[it * 64 + lane] = (uint8_t)m;
      }
      np = gather(exceeds);
      if (np <= kPieces) {
        collect_pieces(np, exceeds);
      } else {
        visit([&](float v, int at) __attribute__((always_inline)) {
          collect(v > t, v, at);
          return n <= kCand;
        });
      }
      if (n <= kCand && n < top) {
        // The first top - n marked values, in order: lane l has kIter pieces.
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kIter; ++i) mine += __popc(tied[lane * kIter + i]);
        int pos = mine;
        for (int off = 1; off < 64; off <<= 1) {
          const int o = __shfl_up(pos, off, 64);
          if (lane >= off) pos += o;
        }
        pos += n - mine;
        for (int i = 0; i < kIter && pos < top; ++i) {
          for (uint32_t w = tied[lane * kIter + i]; w != 0 && pos < top; w &= w - 1, ++pos)
            best[pos] = key_of(t, (uint32_t)(base + (lane * kIter + i) * kVec + __ffs((int)w) - 1));
        }
      }
    }
    if (n <= kCand) {
      wave_order();
      rank_keys<64>(cand, n, top, best);
    } else {
      // Many different values above t (a chunk whose large values share few
      // lanes): one maximum of the wave after the other.
      uint64_t last = ~0ull;
      for (int r = 0; r < top && last != 0; ++r) {
        uint64_t k = 0;
        visit([&](float v, int at) __attribute__((always_inline)) {
          const uint64_t c = v >= t ? key_of(v, (uint32_t)(base + at)) : 0;
          if (c < last) k = max_u64(k, c);
          return true;
        });
        last = wave_max_key(k);
        if (lane == 0) best[r] = last;
      }
    }
    wave_order();
  }
  if (chunks == 1) {
    write_row<T, 64>(z, V, row, st, best, tokens, ntok, top, lp, lse, ent, top_ids, top_lp);
    return;
  }
  if (lane == 0) stats[u] = st;
  if (lane < top) keys[(int64_t)u * top + lane] = best[lane];
}

// Joins the chunks of one row.  Keys below a bound that at least `top` keys
// reach are passed over: of fewer than `top` chunks, the least of the chunks'
// q-th keys, q = ceil(top / chunks); of more, one that `top` of 64 group maxima
// of the chunks' first keys reach.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void logprobs_join_kernel(
    const T* __restrict__ logits, int64_t ld, int64_t V, int chunks, int top, const Stats* __restrict__ stats,
    const uint64_t* __restrict__ keys, const int64_t* __restrict__ tokens, int64_t ntok, float* __restrict__ lp,
    float* __restrict__ lse, float* __restrict__ ent, int64_t* __restrict__ top_ids, float* __restrict__ top_lp) {
  constexpr int kWaves = NT / 64;
  __shared__ float tmax[NT];
  __shared__ float heads[NT];
  __shared__ float redS[kWaves], redW[kWaves];
  __shared__ uint64_t redk[kWaves];
  __shared__ uint64_t cand[kJoinCand];
  __shared__ uint64_t best[PRISM_TOP_MAX];
  __shared__ int ncand;
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Stats* sr = stats + row * chunks;
  const uint64_t* kr = keys + row * chunks * top;
  const bool few = chunks < top;
  const int q = few ? (top + chunks - 1) / chunks : 1;
  const int64_t n = (int64_t)chunks * top;
  // This thread's first chunk and keys, and the bound's part of its chunks.
  Stats s0{kNegInf, 0.0f, 0.0f};
  float m = kNegInf, head = few ? -kNegInf : kNegInf;
  uint64_t k0[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = (int64_t)threadIdx.x + i * NT;
    k0[i] = at < n ? kr[at] : 0;
  }
  for (int c = threadIdx.x; c < chunks; c += NT) {
    const Stats s = sr[c];
    if (c == (int)threadIdx.x) s0 = s;
    m = __builtin_elementwise_maximum(m, s.m);
    if (top > 0) {
      const uint64_t k = kr[(int64_t)c * top + q - 1];
      const float h = k ? value_of(k) : kNegInf;
      head = few ? fminf(head, h) : fmaxf(head, h);
    }
  }
  tmax[threadIdx.x] = m;
  heads[threadIdx.x] = head;
  if (threadIdx.x == 0) ncand = 0;
  if ((int)threadIdx.x < top) best[threadIdx.x] = 0;
  __syncthreads();
  float g = tmax[lane], h = heads[lane];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    g = __builtin_elementwise_maximum(g, tmax[lane + 64 * i]);
    h = few ? fminf(h, heads[lane + 64 * i]) : fmaxf(h, heads[lane + 64 * i]);
  }
  Stats st;
  st.m = wave_max(g);
  float bound = kLowest;
  if (top > 0) bound = fmaxf(few ? wave_min(h) : kth_of_wave(h, wave_max(h), top), kLowest);
  const float b = base_of(st.m);
  float S = 0.0f, W = 0.0f;
  for (int c = threadIdx.x; c < chunks; c += NT) {
    const Stats s = c == (int)threadIdx.x ? s0 : sr[c];
    const float t = log2_term(s.m - b);  // sums of an empty chunk are 0
    const float e = __builtin_amdgcn_exp2f(t);
    S = __builtin_fmaf(e, s.S, S);
    W = __builtin_fmaf(e, __builtin_fmaf(t, s.S, s.W), W);
  }
  S = wave_sum(S);
  W = wave_sum(W);
  if (lane == 0) {
    redS[wave] = S;
    redW[wave] = W;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (k0[i] != 0 && value_of(k0[i]) >= bound) {
      const int at = atomicAdd(&ncand, 1);
      if (at < kJoinCand) cand[at] = k0[i];
    }
  }
  for (int64_t i = threadIdx.x + 4 * NT; i < n; i += NT) {
    const uint64_t k = kr[i];
    if (k != 0 && value_of(k) >= bound) {
      const int at = atomicAdd(&ncand, 1);
      if (at < kJoinCand) cand[at] = k;
    }
  }
  __syncthreads();
  st.S = redS[0];
  st.W = redW[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    st.S += redS[i];
    st.W += redW[i];
  }
  if (ncand <= kRankCand || (ncand <= kJoinCand && chunks > 64)) {
    rank_keys<NT>(cand, ncand, top, best);
  } else if (chunks <= 64 && n <= kJoinCand) {
    // Many keys near the bound (chunks masked to one value): the chunks' sorted
    // keys in LDS, merged by one wave with a chunk per lane.
    __syncthreads();
    for (int i = threadIdx.x; i < (int)n; i += NT) cand[i] = kr[i];
    __syncthreads();
    if (wave == 0) {
      int at = lane * top, left = lane < chunks ? top : 0;
      uint64_t head = left > 0 ? cand[at] : 0;
      for (int r = 0; r < top; ++r) {
        const uint64_t k = wave_max_key(head);
        if (lane == 0) best[r] = k;
        if (k == 0) break;  // best is 0 from here on
        if (head == k) head = --left > 0 ? cand[++at] : 0;
      }
    }
  } else {
    uint64_t last = ~0ull;
    for (int r = 0; r < top && last != 0; ++r) {
      uint64_t k = 0;
      for (int64_t i = threadIdx.x; i < n; i += NT)
        if (kr[i] < last) k = max_u64(k, kr[i]);
      last = block_max_key<NT>(k, redk);
      if (threadIdx.x == 0) best[r] = last;
    }
  }
  __syncthreads();
  write_row<T, NT>(logits + row * ld, V, row, st, best, tokens, ntok, top, lp, lse, ent, top_ids, top_lp);
}

// Threads of a workgroup.  Few chunks: a wave each, to have them on as many CUs.
int chunk_threads(int64_t total) { return total <= 1024 ? 64 : 256; }
// A wave per row while its lanes hold a few keys each (2048 rows of 104 keys:
// 10.5 us with four waves, 7).
int join_threads(int64_t chunks, int top) { return chunks <= 64 && chunks * top <= 256 ? 64 : 256; }

template <typename T>
int launch(const void* logits, int64_t ld, const int64_t* tokens, int64_t ntok, int top, float* lp, float* lse,
           float* ent, int64_t* top_ids, float* top_lp, void* ws, int64_t M, int64_t V, hipStream_t st) {
  const int chunks = (int)((V + kChunk - 1) / kChunk);
  const T* z = static_cast<const T*>(logits);
  uint64_t* keys = static_cast<uint64_t*>(ws);  // 8-byte entries first
  Stats* stats = reinterpret_cast<Stats*>(keys + (chunks > 1 ? M * chunks * top : 0));
  const unsigned total = (unsigned)(M * chunks);
  if (chunk_threads(total) == 64)
    logprobs_chunk_kernel<T, 1><<<total, 64, 0, st>>>(z, ld, V, total, chunks, top, stats, keys, tokens, ntok, lp, lse,
                                                      ent, top_ids, top_lp);
  else
    logprobs_chunk_kernel<T, 4><<<(total + 3) / 4, 256, 0, st>>>(z, ld, V, total, chunks, top, stats, keys, tokens, ntok,
                                                                 lp, lse, ent, top_ids, top_lp);
  if (chunks > 1 && join_threads(chunks, top) == 64)
    logprobs_join_kernel<T, 64><<<(unsigned)M, 64, 0, st>>>(z, ld, V, chunks, top, stats, keys, tokens, ntok, lp, lse, ent,
                                                            top_ids, top_lp);
  else if (chunks > 1)
    logprobs_join_kernel<T, 256><<<(unsigned)M, 256, 0, st>>>(z, ld, V, chunks, top, stats, keys, tokens, ntok, lp, lse,
                                                              ent, top_ids, top_lp);
  return launch_status();
}

}  // namespace

// Workspace: the chunks' keys and statistics; none when a row is one chunk.
int64_t token_logprobs_bytes(int64_t M, int64_t V, int top) {
  const int64_t chunks = (V + kChunk - 1) / kChunk;
  return chunks > 1 ? M * chunks * (8 * (int64_t)top + (int64_t)sizeof(Stats)) : 0;
}

int64_t token_logprobs_threads(int64_t M, int64_t V, int top) {
  const int64_t chunks = (V + kChunk - 1) / kChunk, total = M * chunks;
  const int waves = chunk_threads(total) / 64;
  const int64_t first = (total + waves - 1) / waves * (64 * waves);
  const int64_t second = chunks > 1 ? M * join_threads(chunks, top) : 0;
  return first > second ? first : second;
}

int launch_token_logprobs(const void* logits, int type, int64_t ld, const int64_t* tokens, int64_t ntok, int top,
                          float* lp, float* lse, float* ent, int64_t* top_ids, float* top_lp, void* ws, int64_t M,
                          int64_t V, hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch<float>(logits, ld, tokens, ntok, top, lp, lse, ent, top_ids, top_lp, ws, M, V, st);
  if (type == PRISM_TYPE_F16) return launch<_Float16>(logits, ld, tokens, ntok, top, lp, lse, ent, top_ids, top_lp, ws, M, V, st);
  return launch<__bf16>(logits, ld, tokens, ntok, top, lp, lse, ent, top_ids, top_lp, ws, M, V, st);
}

}  // namespace prism
