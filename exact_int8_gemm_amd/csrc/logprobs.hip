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
// workgroup each, so a row's sums are always added in the same order.  A chunk
// is read once and stays in registers: maximum, sums, and its `top` largest
// values; a second kernel joins the chunks of a row.
//
// Top values: every thread's maximum goes to LDS; lane l takes the maximum
// of the threads l, l + 64, ..., and the top-th largest of these 64 group
// maxima is a value that at least `top` values of the chunk reach.  Only
// values that reach it (usually a few more than `top`) are collected and
// ranked, by value and then by index, as one 64-bit key each.  When too many
// values tie there (a chunk masked to one finite value), `top` rounds of a
// workgroup-wide maximum find them instead.
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
constexpr float kLog2E = 0x1.715476p+0f;
constexpr float kNegInf = -__builtin_inff();
// Stands in for z - m = -inf where it multiplies a probability of 0.
constexpr float kFloor = -1e30f;

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

// z - m with m = -inf (nothing in the row or chunk) taken as 0.
__device__ inline float base_of(float m) { return m == kNegInf ? 0.0f : m; }
__device__ inline float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2E); }

__device__ inline uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ inline uint64_t shfl_xor_u64(uint64_t v, int off) {
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, off, 64);
  const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), off, 64);
  return ((uint64_t)hi << 32) | lo;
}

// Sum over the workgroup, the same bits in every thread.
template <int NT>
__device__ inline float block_sum(float v, float* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s += lds[i];
  __syncthreads();
  return s;
}

template <int NT>
__device__ inline float block_max(float v, float* lds) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s = fmaxf(s, lds[i]);
  __syncthreads();
  return s;
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
    if (ent) ent[row] = bad ? nan : empty ? 0.0f : ls - st.W / st.S;
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
  __shared__ float red[kThreads / 64];
  __shared__ uint64_t redk[kThreads / 64];
  __shared__ float tmax[kThreads];
  __shared__ uint64_t cand[kCand];
  __shared__ uint64_t best[PRISM_TOP_MAX];
  __shared__ int ncand;
  const int64_t row = blockIdx.x / (unsigned)chunks;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int64_t base = (int64_t)chunk * kChunk;
  const T* z = logits + row * ld;

  // Values at base + (it kThreads + thread) kVec + e.  A row may start at any
  // element, so the 16-byte loads are unaligned ones.
  float v[kPerThread];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int64_t at = base + ((int64_t)it * kThreads + threadIdx.x) * kVec;
    T raw[kVec];
    if (at + kVec <= V) {
      __builtin_memcpy(raw, z + at, 16);
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[it * kVec + e] = to_float(raw[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[it * kVec + e] = at + e < V ? to_float(z[at + e]) : kNegInf;
    }
  }
  float mt = kNegInf;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) mt = fmaxf(mt, v[i]);
  tmax[threadIdx.x] = mt;
  if (threadIdx.x == 0) ncand = 0;
  if (threadIdx.x < top) best[threadIdx.x] = 0;
  Stats st;
  st.m = block_max<kThreads>(mt, red);
  const float b = base_of(st.m);
  float S = 0.0f, W = 0.0f;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const float d = v[i] - b;
    const float e = exp_of(d);
    S += e;
    W = __builtin_fmaf(e, fmaxf(d, kFloor), W);
  }
  st.S = block_sum<kThreads>(S, red);
  st.W = block_sum<kThreads>(W, red);

  if (top > 0) {
    // Top-th largest of the 64 group maxima: the largest value that fewer
    // than `top` groups exceed.
    const int lane = threadIdx.x & 63;
    float g = tmax[lane];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) g = fmaxf(g, tmax[lane + 64 * i]);
    int above = 0;
    for (int i = 0; i < 64; ++i)
      above += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g), i)) > g ? 1 : 0;
    float t = above < top ? g : -kNegInf;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) t = fminf(t, __shfl_xor(t, off, 64));
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (v[i] >= t && v[i] > kNegInf) {
        const int at = atomicAdd(&ncand, 1);
        const int64_t idx = base + ((int64_t)(i / kVec) * kThreads + threadIdx.x) * kVec + i % kVec;
        if (at < kCand) cand[at] = key_of(v[i], (uint32_t)idx);
      }
    }
    __syncthreads();
    const int n = ncand;
    if (n <= kCand) {
      rank_keys<kThreads>(cand, n, top, best);
    } else {
      uint64_t last = ~0ull;
      for (int r = 0; r < top && last != 0; ++r) {
        uint64_t k = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          const int64_t idx = base + ((int64_t)(i / kVec) * kThreads + threadIdx.x) * kVec + i % kVec;
          const uint64_t c = v[i] > kNegInf ? key_of(v[i], (uint32_t)idx) : 0;
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

// Joins the chunks of one row.
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void logprobs_join_kernel(
    const T* __restrict__ logits, int64_t ld, int64_t V, int chunks, int top, const Stats* __restrict__ stats,
    const uint64_t* __restrict__ keys, const int64_t* __restrict__ tokens, int64_t ntok, float* __restrict__ lp,
    float* __restrict__ lse, float* __restrict__ ent, int64_t* __restrict__ top_ids, float* __restrict__ top_lp) {
  __shared__ float red[kJoinThreads / 64];
  __shared__ uint64_t redk[kJoinThreads / 64];
  __shared__ uint64_t cand[kJoinCand];
  __shared__ uint64_t best[PRISM_TOP_MAX];
  const int64_t row = blockIdx.x;
  const Stats* sr = stats + row * chunks;
  const uint64_t* kr = keys + row * chunks * top;
  if ((int)threadIdx.x < top) best[threadIdx.x] = 0;
  float m = kNegInf;
  for (int c = threadIdx.x; c < chunks; c += kJoinThreads) m = fmaxf(m, sr[c].m);
  Stats st;
  st.m = block_max<kJoinThreads>(m, red);
  const float b = base_of(st.m);
  float S = 0.0f, W = 0.0f;
  for (int c = threadIdx.x; c < chunks; c += kJoinThreads) {
    const Stats s = sr[c];
    const float d = fmaxf(s.m - b, kFloor);  // sums of an empty chunk are 0
    const float e = exp_of(d);
    S = __builtin_fmaf(e, s.S, S);
    W = __builtin_fmaf(e, __builtin_fmaf(d, s.S, s.W), W);
  }
  st.S = block_sum<kJoinThreads>(S, red);
  st.W = block_sum<kJoinThreads>(W, red);
  const int64_t n = (int64_t)chunks * top;
  if (n <= kJoinCand) {
    for (int i = threadIdx.x; i < (int)n; i += kJoinThreads) cand[i] = kr[i];
    __syncthreads();
    for (int i = threadIdx.x; i < (int)n; i += kJoinThreads) {
      const uint64_t k = cand[i];
      if (k == 0) continue;
      int rank = 0;
      for (int j = 0; j < (int)n; ++j) rank += cand[j] > k ? 1 : 0;
      if (rank < top) best[rank] = k;
    }
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
