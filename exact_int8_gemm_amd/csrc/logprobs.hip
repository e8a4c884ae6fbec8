// Token read-out: log probabilities of given tokens, the entropy and the top
// alternatives of each row of logits (the method's engine answers typed
// questions from the probabilities of given tokens after one forward pass;
// StartLux-Prism README, "Example" and "How it works").
//
// With m = max z, S = sum exp(z - m), W = sum exp(z - m) (z - m):
//   lse = m + log S, logprob(t) = (z_t - m) - log S, entropy = log S - W / S.
// Both terms of the entropy are >= 0, so nothing cancels.  m, S and W are
// fp32; exp is one v_exp_f32 of (z - m) log2(e), whose error (|z - m| 2^-24
// relative) is largest where the term itself vanishes.  (z log2(e) - m log2(e)
// as one fma would save an instruction and be off by |z| 2^-24 in every term.)
//
// The vocabulary axis is cut into chunks of kChunk values whatever M is, one
// workgroup each, so a row's sums are always added in the same order.  A chunk
// is read once and stays in registers: maximum, sums, and its `top` largest
// values; a second kernel joins the chunks of a row.
//
// Top values: every thread's maximum goes to LDS; lane l takes the maximum
// of the threads l, l + 64, ..., and the top-th largest of these 64 group
// maxima is a value that at least `top` values of the chunk reach.  Only
// values that reach it (usually a few more than `top`) are collected and
// ranked, by value and then by index, as one 64-bit key each.  When too many
// values tie there (a chunk masked to one finite value), the larger ones are
// ranked and the tied ones marked in a bit per value, of which the first are
// taken.
//
#include "../../include/prism.h"
#include "prism_internal.h"

namespace prism {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 32;
constexpr int kChunk = kThreads * kPerThread;
constexpr int kCand = 512;  // candidates ranked at once
constexpr int kJoinThreads = 256;
constexpr int kJoinCand = 1024;
constexpr float kLowest = -3.402823466e+38f;
constexpr float kLog2E = 0x1.715476p+0f, kLn2 = 0x1.62e430p-1f;
constexpr float kNegInf = -__builtin_inff();
// Lowest exponent of 2 taken: 2^-200 is 0 in fp32, and unlike -inf it can be
// multiplied by that.
constexpr float kFloor = -200.0f;

struct Stats {
  float m, S, W;
};

// Keys order values first, then lower indices; 0 is below every key of a
// value above -inf.  + 0.0f makes -0 equal to 0.
__device__ inline uint64_t key_of(float v, uint32_t index) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  const uint32_t o = (b >> 31) ? ~b : (b | 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~index;
}
__device__ inline float value_of(uint64_t key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __builtin_bit_cast(float, (o >> 31) ? (o & 0x7fffffffu) : ~o);
}
__device__ inline uint32_t index_of(uint64_t key) { return ~(uint32_t)key; }

template <typename T>
__device__ inline float to_float(T v) {
  return (float)v;
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
  return wave_reduce(v, kNegInf, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float wave_min(float v) {
  return wave_reduce(v, -kNegInf, [](float a, float b) { return fminf(a, b); });
}
__device__ inline float wave_sum(float v) {
  return wave_reduce(v, 0.0f, [](float a, float b) { return a + b; });
}

// The top-th largest of the lanes' values (top <= 64): the least value that
// fewer than `top` lanes exceed.
__device__ inline float kth_of_wave(float g, int top) {
  int above = 0;
#pragma unroll 16
  for (int i = 0; i < 64; ++i)
    above += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g), i)) > g ? 1 : 0;
  return wave_min(above < top ? g : -kNegInf);
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
  for (int i = threadIdx.x; i < n; i += NT) {
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
  if (threadIdx.x == 0) {
    if (lse) lse[row] = bad ? nan : empty ? kNegInf : base + ls;
    if (ent) ent[row] = bad ? nan : empty ? 0.0f : ls - st.W * kLn2 / st.S;
  }
  for (int64_t i = threadIdx.x; i < ntok; i += NT) {
    const int64_t t = tokens[row * ntok + i];
    float r = nan;
    if (t >= 0 && t < V && !bad) r = empty ? kNegInf : (to_float(z[t]) - base) - ls;
    lp[row * ntok + i] = r;
  }
  for (int i = threadIdx.x; i < top; i += NT) {
    const uint64_t k = keys[i];
    float r = kNegInf;
    if (k != 0 && !empty && !bad) r = (value_of(k) - base) - ls;
    top_lp[row * top + i] = bad ? nan : r;
    top_ids[row * top + i] = (bad || r == kNegInf) ? -1 : (int64_t)index_of(k);
  }
}

// One chunk of one row: statistics and sorted top keys into stats[row][chunk]
// and keys[row][chunk][top]; or, if the row is one chunk, the row's results.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_chunk_kernel(
    const T* __restrict__ logits, int64_t ld, int64_t V, int chunks, int top, Stats* __restrict__ stats,
    uint64_t* __restrict__ keys, const int64_t* __restrict__ tokens, int64_t ntok, float* __restrict__ lp,
    float* __restrict__ lse, float* __restrict__ ent, int64_t* __restrict__ top_ids, float* __restrict__ top_lp) {
  constexpr int kVec = 16 / (int)sizeof(T);
  constexpr int kIter = kPerThread / kVec;
  constexpr int kWaves = kThreads / 64;
  constexpr int kGroups = kPerThread / 8;
  __shared__ float tmax[kThreads];
  __shared__ float redS[kWaves], redW[kWaves];
  __shared__ float lthr;
  __shared__ uint64_t redk[kWaves];
  __shared__ uint64_t cand[kCand];
  __shared__ uint64_t best[PRISM_TOP_MAX];
  __shared__ uint32_t tied[kChunk / 32];
  __shared__ int ncand;
  const int64_t row = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int64_t base = (int64_t)chunk * kChunk;
  const T* z = logits + row * ld;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  // Value i of this thread is value place(i) of the chunk: pieces of kVec
  // consecutive ones.  A row may start at any element, so the 16-byte loads
  // are unaligned ones.
  auto place = [&](int i) { return ((i / kVec) * kThreads + (int)threadIdx.x) * kVec + i % kVec; };
  float v[kPerThread];
  const int64_t left = V - base;  // values from the chunk's first to the row's end
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int at = place(it * kVec);
    T raw[kVec];
    if (at + kVec <= left) {
      __builtin_memcpy(raw, z + base + at, 16);
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[it * kVec + e] = to_float(raw[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[it * kVec + e] = at + e < left ? to_float(z[base + at + e]) : kNegInf;
    }
  }
  float gm[kGroups], mt = kNegInf;  // maxima of eight values each (a NaN is passed over), and of all
#pragma unroll
  for (int a = 0; a < kGroups; ++a) {
    gm[a] = v[8 * a];
#pragma unroll
    for (int e = 1; e < 8; ++e) gm[a] = fmaxf(gm[a], v[8 * a + e]);
    mt = fmaxf(mt, gm[a]);
  }
  tmax[threadIdx.x] = mt;
  if (threadIdx.x == 0) ncand = 0;
  if ((int)threadIdx.x < top) best[threadIdx.x] = 0;
  __syncthreads();
  float g = tmax[lane];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) g = fmaxf(g, tmax[lane + 64 * i]);
  Stats st;
  st.m = wave_max(g);
  if (top > 0 && wave == 0) {
    const float t = fmaxf(kth_of_wave(g, top), kLowest);  // -inf is never listed
    if (lane == 0) lthr = t;
  }
  const float b = base_of(st.m);
  float S = 0.0f, W = 0.0f;  // W in powers of 2
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const float t = log2_term(v[i] - b);
    const float e = __builtin_amdgcn_exp2f(t);
    S += e;
    W = __builtin_fmaf(e, t, W);
  }
  S = wave_sum(S);
  W = wave_sum(W);
  if (lane == 0) {
    redS[wave] = S;
    redW[wave] = W;
  }
  __syncthreads();
  st.S = redS[0];
  st.W = redW[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    st.S += redS[i];
    st.W += redW[i];
  }

  if (top > 0) {
    const float t = lthr;
    auto collect = [&](auto&& wanted) __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < kGroups; ++a) {
        if (!wanted(gm[a])) continue;
#pragma unroll
        for (int i = 8 * a; i < 8 * a + 8; ++i) {
          if (!wanted(v[i])) continue;
          const int at = atomicAdd(&ncand, 1);
          if (at < kCand) cand[at] = key_of(v[i], (uint32_t)(base + place(i)));
        }
      }
    };
    collect([&](float x) { return x >= t; });
    __syncthreads();
    int n = ncand;
    if (n > kCand) {
      // Many values tie at t: rank the larger ones, mark the tied ones.
      __syncthreads();
      if (threadIdx.x == 0) ncand = 0;
      for (int i = threadIdx.x; i < kChunk / 32; i += kThreads) tied[i] = 0;
      __syncthreads();
      collect([&](float x) { return x > t; });
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) m |= v[it * kVec + e] == t ? 1u << e : 0u;
        const int at = place(it * kVec);
        if (m) atomicOr(&tied[at / 32], m << (at % 32));
      }
      __syncthreads();
      n = ncand;
      if (n <= kCand && n < top && wave == 0) {
        // The first top - n marked values, in order: lane l has kPer words.
        constexpr int kPer = kChunk / 32 / 64;
        int mine = 0;
        for (int i = 0; i < kPer; ++i) mine += __popc(tied[lane * kPer + i]);
        int pos = mine;
        for (int off = 1; off < 64; off <<= 1) {
          const int o = __shfl_up(pos, off, 64);
          if (lane >= off) pos += o;
        }
        pos += n - mine;
        for (int i = 0; i < kPer && pos < top; ++i) {
          for (uint32_t w = tied[lane * kPer + i]; w != 0 && pos < top; w &= w - 1, ++pos)
            best[pos] = key_of(t, (uint32_t)(base + (lane * kPer + i) * 32 + __ffs((int)w) - 1));
        }
      }
    }
    if (n <= kCand) {
      rank_keys<kThreads>(cand, n, top, best);
    } else {
      // Many different values above t (a chunk whose large values share few
      // groups): one maximum of the workgroup after the other.
      uint64_t last = ~0ull;
      for (int r = 0; r < top && last != 0; ++r) {
        uint64_t k = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          const uint64_t c = v[i] > kNegInf ? key_of(v[i], (uint32_t)(base + place(i))) : 0;
          if (c < last) k = max_u64(k, c);
        }
        last = block_max_key<kThreads>(k, redk);
        if (threadIdx.x == 0) best[r] = last;
      }
    }
    __syncthreads();
  }
  if (chunks == 1) {
    write_row<T, kThreads>(z, V, row, st, best, tokens, ntok, top, lp, lse, ent, top_ids, top_lp);
    return;
  }
  const int64_t slot = row * chunks + chunk;
  if (threadIdx.x == 0) stats[slot] = st;
  if ((int)threadIdx.x < top) keys[slot * top + threadIdx.x] = best[threadIdx.x];
}

// Joins the chunks of one row.  Keys below a bound that at least `top` keys
// reach are passed over: of fewer than `top` chunks, the least of the chunks'
// q-th keys, q = ceil(top / chunks); of more, the top-th largest of 64 group
// maxima of the chunks' first keys.
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void logprobs_join_kernel(
    const T* __restrict__ logits, int64_t ld, int64_t V, int chunks, int top, const Stats* __restrict__ stats,
    const uint64_t* __restrict__ keys, const int64_t* __restrict__ tokens, int64_t ntok, float* __restrict__ lp,
    float* __restrict__ lse, float* __restrict__ ent, int64_t* __restrict__ top_ids, float* __restrict__ top_lp) {
  constexpr int kWaves = kJoinThreads / 64;
  __shared__ float tmax[kJoinThreads];
  __shared__ float heads[kJoinThreads];
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
    const int64_t at = (int64_t)threadIdx.x + i * kJoinThreads;
    k0[i] = at < n ? kr[at] : 0;
  }
  for (int c = threadIdx.x; c < chunks; c += kJoinThreads) {
    const Stats s = sr[c];
    if (c == (int)threadIdx.x) s0 = s;
    m = fmaxf(m, s.m);
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
    g = fmaxf(g, tmax[lane + 64 * i]);
    h = few ? fminf(h, heads[lane + 64 * i]) : fmaxf(h, heads[lane + 64 * i]);
  }
  Stats st;
  st.m = wave_max(g);
  float bound = kLowest;
  if (top > 0) bound = fmaxf(few ? wave_min(h) : kth_of_wave(h, top), kLowest);
  const float b = base_of(st.m);
  float S = 0.0f, W = 0.0f;
  for (int c = threadIdx.x; c < chunks; c += kJoinThreads) {
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
  for (int64_t i = threadIdx.x + 4 * kJoinThreads; i < n; i += kJoinThreads) {
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
  if (ncand <= kJoinCand) {
    rank_keys<kJoinThreads>(cand, ncand, top, best);
  } else {
    uint64_t last = ~0ull;
    for (int r = 0; r < top && last != 0; ++r) {
      uint64_t k = 0;
      for (int64_t i = threadIdx.x; i < n; i += kJoinThreads)
        if (kr[i] < last) k = max_u64(k, kr[i]);
      last = block_max_key<kJoinThreads>(k, redk);
      if (threadIdx.x == 0) best[r] = last;
    }
  }
  __syncthreads();
  write_row<T, kJoinThreads>(logits + row * ld, V, row, st, best, tokens, ntok, top, lp, lse, ent, top_ids, top_lp);
}

template <typename T>
int launch(const void* logits, int64_t ld, const int64_t* tokens, int64_t ntok, int top, float* lp, float* lse,
           float* ent, int64_t* top_ids, float* top_lp, void* ws, int64_t M, int64_t V, hipStream_t st) {
  const int chunks = (int)((V + kChunk - 1) / kChunk);
  const T* z = static_cast<const T*>(logits);
  uint64_t* keys = static_cast<uint64_t*>(ws);  // 8-byte entries first
  Stats* stats = reinterpret_cast<Stats*>(keys + (chunks > 1 ? M * chunks * top : 0));
  logprobs_chunk_kernel<T><<<(unsigned)(M * chunks), kThreads, 0, st>>>(z, ld, V, chunks, top, stats, keys, tokens, ntok,
                                                                        lp, lse, ent, top_ids, top_lp);
  if (chunks > 1)
    logprobs_join_kernel<T><<<(unsigned)M, kJoinThreads, 0, st>>>(z, ld, V, chunks, top, stats, keys, tokens, ntok, lp,
                                                                  lse, ent, top_ids, top_lp);
  return launch_status();
}

}  // namespace

// Workspace: the chunks' keys and statistics; none when a row is one chunk.
int64_t token_logprobs_bytes(int64_t M, int64_t V, int top) {
  const int64_t chunks = (V + kChunk - 1) / kChunk;
  return chunks > 1 ? M * chunks * (8 * (int64_t)top + (int64_t)sizeof(Stats)) : 0;
}

int64_t token_logprobs_groups(int64_t M, int64_t V) { return M * ((V + kChunk - 1) / kChunk); }

int launch_token_logprobs(const void* logits, int type, int64_t ld, const int64_t* tokens, int64_t ntok, int top,
                          float* lp, float* lse, float* ent, int64_t* top_ids, float* top_lp, void* ws, int64_t M,
                          int64_t V, hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch<float>(logits, ld, tokens, ntok, top, lp, lse, ent, top_ids, top_lp, ws, M, V, st);
  if (type == PRISM_TYPE_F16) return launch<_Float16>(logits, ld, tokens, ntok, top, lp, lse, ent, top_ids, top_lp, ws, M, V, st);
  return launch<__bf16>(logits, ld, tokens, ntok, top, lp, lse, ent, top_ids, top_lp, ws, M, V, st);
}

}  // namespace prism
