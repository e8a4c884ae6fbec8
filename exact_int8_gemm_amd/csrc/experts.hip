// Routing of a mixture-of-experts layer, and the weighted sum behind it: the
// parts around the grouped products (gemm_fp8_grouped.hip) that make them a layer
// of the quantized model (StartLux-Prism README, "Why StartLux-Prism": a row's
// result does not depend on what it is batched with).
//
// Routing, per token: the `top` experts of largest key, the lower index first
// among equal keys, their weights, and a counting sort of all choices by expert
// that keeps the order of the tokens.  The key is the logit itself, or with a bias
// the score plus the bias in 64 bits: sums that round to the same 64 bits (sigmoids of
// logits above 37, scores far below a bias's last bit) are equal keys.  One wave takes one
// token: lane l holds experts V l ... V l + V - 1.
//
// The sort works on 32 tokens at a time.  A token chooses an expert once at the
// most, so an expert's tokens are the bits of one word, set by atomic ors whose
// order does not matter; their number is its population count and a choice's
// rank that of the bits below its own.  One workgroup routes `passes` times 32
// tokens and leaves its counts per expert; a second launch adds up the counts in
// front of each workgroup's and places the choices.
//
// Both are bound by latency: a wave's chain of load, bound, ranking and 64-bit
// exponential, twice, and two dependent launches (8192 x 256 fp32, top 8, with a
// bias: 11.8 + 6.5 us, of which the bytes are 2; 4 x 128: 4.6, one launch).  With a
// bias, 513 to 1024 experts are 16 to a lane, and 22 of its vector registers are spilled
// to 92 bytes of scratch; no other form spills any.
#include <type_traits>

#include "../../include/prism.h"
#include "prism_internal.h"
#include "wave.h"

namespace prism {
namespace {

constexpr int kTokens = 32;       // of a pass: the bits of a word
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxChunks = 512;   // workgroups of a call

struct Route {
  const void* logits;
  int64_t ld;
  const float* bias;
  int score, renormalize;
  float scale;
  int top;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* slots;
  uint16_t* counts;  // [workgroups][pitch_of(E)]
  int M, E, passes;
};

template <int CTRL, int ROWS>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false));
}
// Over the wave, without LDS: shifts within rows of 16 lanes, then row broadcasts.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xf>(v);  // row_shr:1
  v = dpp_max<0x112, 0xf>(v);
  v = dpp_max<0x114, 0xf>(v);
  v = dpp_max<0x118, 0xf>(v);
  v = dpp_max<0x142, 0xa>(v);  // row_bcast:15
  v = dpp_max<0x143, 0xc>(v);  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline uint64_t wave_max(uint64_t k) {
  const uint32_t hi = wave_max((uint32_t)(k >> 32));
  const uint32_t lo = wave_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}
template <int CTRL, int ROWS>
__device__ inline double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ inline double wave_sum(double v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  v = dpp_add<0x143, 0xc>(v);
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ inline int wave_inclusive(int v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off, 64);
    if ((int)(threadIdx.x & 63) >= off) v += o;
  }
  return v;
}

// Order of the values, above 0; + 0 makes -0 equal to 0.
__device__ inline uint32_t order_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ inline uint64_t order_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000u);
}

__device__ inline float of_order(uint32_t o) {
  return __builtin_bit_cast(float, (o >> 31) ? (o & 0x7fffffffu) : ~o);
}

template <typename K>
__device__ inline K readlane(K v, int lane) {
  if constexpr (sizeof(K) == 4) {
    return (K)__builtin_amdgcn_readlane((int)v, lane);
  } else {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return ((uint64_t)hi << 32) | lo;
  }
}

__device__ inline double sigmoid(double z) { return 1.0 / (1.0 + exp(-z)); }
// Scores within 2^-20, for keys that are looked at again: an exponent's argument is
// off by 2^-23 |z|, which moves a score by that times |z| exp(-|z|) at the most.  A
// sum with a bias is rounded by 2^-24 of it; kNear is eight times both.
__device__ inline float near_exp(float z) { return __builtin_amdgcn_exp2f(z * 0x1.715476p+0f); }
__device__ inline float near_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + near_exp(-z)); }
constexpr float kNear = 0x1p-17f;

// A wave's LDS: what it ranks, and the choices in their order.
struct Ranked {
  double score[64];
  float z[64];
  uint16_t expert[64];
};

// One token's choice by a wave.  Lane j < top gets choice j (-1: none left) and its weight.
//
// A bound that at least `top` lanes' largest keys reach is found bit by bit.  The
// keys that reach it, a few more than `top`, go to one lane each and are ranked, by
// key and then by index.  With a bias the bound is one on keys in fp32, lowered by
// more than their error, and only what reaches it has its key computed in 64 bits
// (8192 x 256, top 8: that and the ranking for a maximum over the lanes for each
// choice, with all keys in 64 bits, 20 us).  More keys than lanes, in rows of many
// equal or few open ones, are chosen by such maxima.
template <typename T, int V, bool BIAS>
__device__ inline void choose(const Route& a, int row, Ranked& lds, int& id, float& weight) {
  using Key = typename std::conditional<BIAS, uint64_t, uint32_t>::type;
  const int lane = threadIdx.x & 63;
  const T* zp = static_cast<const T*>(a.logits) + (int64_t)row * a.ld + lane * V;
  const float kInf = __builtin_inff();
  float z[V];
  if (a.E == 64 * V) {
    T t[V];
    __builtin_memcpy(t, zp, sizeof(t));  // rows start at any element
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = (float)t[v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = lane * V + v < a.E ? (float)zp[v] : -kInf;
  }
  bool bad = false;
  float most = -kInf;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bad = bad || !(z[v] < kInf);  // NaN or +inf
    most = fmaxf(most, z[v]);
  }
  id = -1;
  weight = 0.0f;
  if (__any(bad)) {
    weight = __builtin_nanf("");
    return;
  }
  const bool softmax = a.score == PRISM_SCORE_SOFTMAX;
  float shift = 0.0f;   // of the softmax
  double total = 1.0;
  if (softmax) {
    const float f = of_order(wave_max(order_of(most)));
    if (f > -kInf) shift = f;
    if (BIAS || !a.renormalize) {
      double mine = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) mine += exp((double)z[v] - (double)shift);
      total = wave_sum(mine);
    }
  }
  auto score_of = [&](float zv) { return softmax ? exp((double)zv - (double)shift) / total : sigmoid((double)zv); };
  auto key_of = [&](float zv, double score, int e) -> Key {
    if constexpr (BIAS) {
      const double k = score + (double)a.bias[e];
      return zv > -kInf && k > -__builtin_inf() ? order_of(k) : 0;
    } else {
      return zv > -kInf ? order_of(zv) : 0;
    }
  };
  // keys in fp32, 0 for what is closed, and the bound on them
  uint32_t near[V], largest = 0;
  const float over = softmax ? 1.0f / (float)total : 1.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    near[v] = z[v] > -kInf ? order_of(z[v]) : 0;
    if constexpr (BIAS) {
      const int e = lane * V + v;
      const float k = (softmax ? near_exp(z[v] - shift) * over : near_sigmoid(z[v])) + (e < a.E ? a.bias[e] : 0.0f);
      near[v] = near[v] && k > -kInf ? order_of(k) : 0;
    }
    largest = max(largest, near[v]);
  }
  // a 16-bit logit's key has nothing of its own in the lowest bits
  constexpr int kLowest = BIAS || sizeof(T) == 4 ? 0 : std::is_same<T, _Float16>::value ? 13 : 16;
  uint32_t bound = 0;
  for (uint32_t bit = 1u << 31; bit >= 1u << kLowest; bit >>= 1) {
    const int reach = __popcll(__ballot(largest >= (bound | bit)));
    if (reach >= a.top) bound |= bit;
    if (reach == a.top) break;
  }
  if (BIAS && bound) {
    const float f = of_order(bound);
    // NaN where f is infinite or of no finite key: all open experts
    const float low = f - (__builtin_fabsf(f) * kNear + kNear);
    bound = low == low ? order_of(low) : 0;
  }
  bound = max(bound, 1u);
  int count = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint64_t in = __ballot(near[v] >= bound);
    const int at = count + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
    if (near[v] >= bound && at < 64) {
      lds.z[at] = z[v];
      lds.expert[at] = (uint16_t)(lane * V + v);
    }
    count += __popcll(in);
  }
  double score = 0.0;
  if (count <= 64) {
    wave_order();
    const bool live = lane < count;
    const float zv = live ? lds.z[lane] : 0.0f;
    const int e = live ? lds.expert[lane] : 0;
    const double sc = score_of(zv);
    const Key key = live ? key_of(zv, sc, e) : 0;
    int rank = 0;
    for (int j = 0; j < count; ++j) {
      const Key other = readlane(key, j);
      const int oe = __builtin_amdgcn_readlane(e, j);
      rank += other > key || (other == key && oe < e) ? 1 : 0;
    }
    wave_order();
    const int chosen = __popcll(__ballot(live && key != 0 && rank < a.top));
    if (live && key != 0 && rank < a.top) {
      lds.score[rank] = sc;
      lds.expert[rank] = (uint16_t)e;
    }
    wave_order();
    if (lane < chosen) {
      score = lds.score[lane];
      id = lds.expert[lane];
    }
    wave_order();
  } else {
    Key key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key_of(z[v], BIAS ? score_of(z[v]) : 0.0, min(lane * V + v, a.E - 1));
    float mine = 0.0f;
    for (int j = 0; j < a.top; ++j) {
      Key local = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) local = key[v] > local ? key[v] : local;
      const Key best = wave_max(local);
      if (best == 0) break;
      const int holder = (int)__builtin_ctzll(__ballot(local == best));
      int which = 0;
      float value = 0.0f;
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == best) {
          which = v;
          value = z[v];
        }
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (lane == holder && v == which) key[v] = 0;
      const int e = holder * V + __builtin_amdgcn_readlane(which, holder);
      const float zv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, value), holder));
      if (lane == j) {
        id = e;
        mine = zv;
      }
    }
    score = id >= 0 ? score_of(mine) : 0.0;
  }
  if (a.renormalize) {
    const double sum = wave_sum(score);
    score = sum > 0.0 ? score / sum : 0.0;
  }
  weight = (float)(score * (double)a.scale);
}

// Experts' counts of a workgroup, whole fours of them.
__host__ __device__ inline int pitch_of(int E) { return (E + 3) / 4 * 4; }
constexpr int kGroups = 32;  // threads that share the workgroups' counts of an expert

// What the workgroups of both launches hold.
struct Shared {
  uint32_t mask[PRISM_EXPERTS_MAX];  // the pass's tokens of each expert
  int base[PRISM_EXPERTS_MAX];       // each expert's next place
  int waves[kWaves];
  uint16_t id[kTokens * PRISM_TOP_MAX];
};

// Exclusive sum of v over the threads.
__device__ inline int block_exclusive(Shared& s, int v) {
  const int in = wave_inclusive(v), wave = (int)threadIdx.x / 64;
  if ((threadIdx.x & 63) == 63) s.waves[wave] = in;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < kWaves; ++w)
    if (w < wave) before += s.waves[w];
  __syncthreads();
  return before + in - v;
}

// The tokens of the pass that starts at `first`, chosen by the waves.
template <typename T, int V, bool BIAS>
__device__ inline void route_pass(const Route& a, Shared& s, Ranked* ranked, int first) {
  const int lane = threadIdx.x & 63, wave = (int)threadIdx.x / 64;
  for (int r = wave; r < kTokens && first + r < a.M; r += kWaves) {
    int id;
    float weight;
    choose<T, V, BIAS>(a, first + r, ranked[wave], id, weight);
    if (lane < a.top) {
      const int64_t at = (int64_t)(first + r) * a.top + lane;
      a.ids[at] = id;
      a.weights[at] = weight;
      s.id[r * a.top + lane] = (uint16_t)id;
      if (id >= 0) atomicOr(&s.mask[id], 1u << r);
    }
  }
}

// Places the choices of the pass: mask, id and base are there.
__device__ inline void place_pass(const Route& a, Shared& s, int first) {
  const int count = min(kTokens, a.M - first) * a.top;
  for (int i = (int)threadIdx.x; i < count; i += kThreads) {
    const int r = i / a.top;
    const uint16_t id = s.id[i];
    int at = -1;
    if (id != 0xffff) {
      at = s.base[id] + __popc(s.mask[id] & ((1u << r) - 1));
      a.rows[at] = first + r;
    }
    a.slots[(int64_t)first * a.top + i] = at;
  }
}

// Offsets from an expert's count in each thread; base starts at them plus `before`.
__device__ inline int start(const Route& a, Shared& s, int total, int before, bool write) {
  const int t = (int)threadIdx.x;
  const int offset = block_exclusive(s, t < a.E ? total : 0);
  if (t < a.E) {
    s.base[t] = offset + before;
    if (write) a.offsets[t] = offset;
    if (t == a.E - 1) {
      s.waves[0] = offset + total;
      if (write) a.offsets[a.E] = offset + total;
    }
  }
  __syncthreads();
  return s.waves[0];
}

// Rows behind the last choice.
__device__ inline void fill_rest(const Route& a, int used) {
  const int64_t all = (int64_t)a.M * a.top;
  for (int64_t i = used + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kThreads)
    a.rows[i] = -1;
}

// ONE: the call has one workgroup and one pass, and needs no second launch.
template <typename T, int V, bool BIAS, bool ONE>
__global__ __launch_bounds__(kThreads) void route_kernel(const Route a) {
  __shared__ Shared s;
  __shared__ Ranked ranked[kWaves];
  const int t = (int)threadIdx.x;
  int count = 0;
  for (int p = 0; p < a.passes; ++p) {
    const int first = ((int)blockIdx.x * a.passes + p) * kTokens;
    s.mask[t] = 0;
    __syncthreads();
    if (first < a.M) route_pass<T, V, BIAS>(a, s, ranked, first);
    __syncthreads();
    count += __popc(s.mask[t]);
  }
  if constexpr (ONE) {
    const int used = start(a, s, count, 0, true);
    place_pass(a, s, 0);
    fill_rest(a, used);
  } else {
    if (t < pitch_of(a.E)) a.counts[(int64_t)blockIdx.x * pitch_of(a.E) + t] = t < a.E ? (uint16_t)count : 0;
  }
}

// Thread (g, c) adds up experts 4 c .. 4 c + 3 of workgroups g, g + groups, ...: of
// those in front of this one, and of all.
__global__ __launch_bounds__(kThreads) void place_kernel(const Route a) {
  __shared__ Shared s;
  __shared__ __attribute__((aligned(16))) int part[2][4 * kThreads];
  const int t = (int)threadIdx.x, chunk = (int)blockIdx.x, chunks = (int)gridDim.x;
  const int pitch = pitch_of(a.E), columns = pitch / 4, groups = min(kThreads / columns, kGroups);
  const int g = t / columns, c = t - g * columns;
  if (g < groups) {
    v4i before{0, 0, 0, 0}, total{0, 0, 0, 0};
    const uint16_t* p = a.counts + 4 * c;
    constexpr int kDeep = 8;
    for (int w0 = g; w0 < chunks; w0 += groups * kDeep) {
      v2i n[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int w = w0 + groups * i;
        n[i] = w < chunks ? *reinterpret_cast<const v2i*>(p + (int64_t)w * pitch) : v2i{0, 0};
      }
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const v4i four{n[i][0] & 0xffff, (int)((uint32_t)n[i][0] >> 16), n[i][1] & 0xffff, (int)((uint32_t)n[i][1] >> 16)};
        total += four;
        if (w0 + groups * i < chunk) before += four;
      }
    }
    *reinterpret_cast<v4i*>(&part[0][g * pitch + 4 * c]) = before;
    *reinterpret_cast<v4i*>(&part[1][g * pitch + 4 * c]) = total;
  }
  __syncthreads();
  int before = 0, total = 0;
  if (t < a.E) {
    for (int i = 0; i < groups; ++i) {
      before += part[0][i * pitch + t];
      total += part[1][i * pitch + t];
    }
  }
  const int used = start(a, s, total, before, chunk == 0);
  for (int p = 0; p < a.passes; ++p) {
    const int first = (chunk * a.passes + p) * kTokens;
    if (first >= a.M) break;
    s.mask[t] = 0;
    __syncthreads();
    const int count = min(kTokens, a.M - first) * a.top;
    for (int i = t; i < count; i += kThreads) {
      const int id = a.ids[(int64_t)first * a.top + i];
      s.id[i] = (uint16_t)id;
      if (id >= 0) atomicOr(&s.mask[id], 1u << (i / a.top));
    }
    __syncthreads();
    place_pass(a, s, first);
    __syncthreads();
    s.base[t] += __popc(s.mask[t]);
  }
  fill_rest(a, used);
}

int passes_of(int64_t M) {
  const int64_t most = (int64_t)kTokens * kMaxChunks;
  return M > most ? (int)((M + most - 1) / most) : 1;
}
int chunks_of(int64_t M) {
  const int64_t per = (int64_t)kTokens * passes_of(M);
  return (int)((M + per - 1) / per);
}

template <typename T, int V, bool BIAS>
int launch_experts(const Route& a, hipStream_t st) {
  const int chunks = chunks_of(a.M);
  if (chunks == 1 && a.passes == 1) {
    route_kernel<T, V, BIAS, true><<<1, kThreads, 0, st>>>(a);
    return launch_status();
  }
  route_kernel<T, V, BIAS, false><<<chunks, kThreads, 0, st>>>(a);
  place_kernel<<<chunks, kThreads, 0, st>>>(a);
  return launch_status();
}

template <typename T, bool BIAS>
int launch_values(const Route& a, hipStream_t st) {
  if (a.E <= 64) return launch_experts<T, 1, BIAS>(a, st);
  if (a.E <= 128) return launch_experts<T, 2, BIAS>(a, st);
  if (a.E <= 256) return launch_experts<T, 4, BIAS>(a, st);
  if (a.E <= 512) return launch_experts<T, 8, BIAS>(a, st);
  return launch_experts<T, 16, BIAS>(a, st);
}

template <typename T>
int launch_bias(const Route& a, hipStream_t st) {
  return a.bias ? launch_values<T, true>(a, st) : launch_values<T, false>(a, st);
}

// ------------------------------------------------------------ weighted sum

// y[m] = add[m] + sum over j ascending of weights[m][j] x[slots[m][j]], in fp32.
// Bound by reading x: a thread takes eight columns of a row and has up to eight
// rows of x on their way.  Rows of 512 columns or more have workgroups of their own
// (8192 x 8 of 5120 bf16, us: 178, threads numbered through all rows 197).  An x
// larger than the cache behind the L2s is read, and y written, past it (that one 166;
// but 3000 x 6 of 1021, 37 MB just written, 14.5, past the cache 18.9).
constexpr int kAhead = 8;
constexpr int64_t kCacheBytes = (int64_t)256 << 20;

template <bool STREAM, typename T>
__device__ inline void load_part(const T* p, int n, float* v) {
  typedef T v8 __attribute__((ext_vector_type(8), aligned(sizeof(T))));  // rows start anywhere
  if (n >= 8) {
    const v8* p8 = reinterpret_cast<const v8*>(p);
    const v8 t = STREAM ? __builtin_nontemporal_load(p8) : *p8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? (float)p[e] : 0.0f;
  }
}

// ROW: a workgroup's threads are in one row, whose slots and weights are then
// scalars.
template <typename T, typename OUT, bool ROW, bool STREAM>
__global__ __launch_bounds__(1024) void combine_kernel(const T* __restrict__ x, const float* __restrict__ weights,
                                                      const int32_t* __restrict__ slots, const OUT* add, OUT* y,
                                                      int R, int M, int top, int N, uint32_t per_row, uint32_t parts) {
  int m, n;
  if (ROW) {
    m = (int)(blockIdx.x / parts);
    n = (int)(blockIdx.x % parts * blockDim.x + threadIdx.x) * 8;
    if (n >= N) return;
  } else {
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;
    m = (int)(at / per_row);
    n = (int)(at % per_row) * 8;
    if (m >= M) return;
  }
  float acc[8];
  if (add) {
    load_part<STREAM>(add + (int64_t)m * N + n, N - n, acc);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  }
  for (int j0 = 0; j0 < top; j0 += kAhead) {
    float w[kAhead], v[kAhead][8];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool in = j0 + j < top;
      const int64_t i = (int64_t)m * top + (in ? j0 + j : 0);
      const int slot = in ? slots[i] : -1;
      w[j] = in ? weights[i] : 0.0f;
      if ((uint32_t)slot < (uint32_t)R) {
        load_part<STREAM>(x + (int64_t)slot * N + n, N - n, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j >= top) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(w[j], v[j][e], acc[e]);
    }
  }
  OUT* yp = y + (int64_t)m * N + n;
  if (N - n >= 8) {
    typedef OUT v8 __attribute__((ext_vector_type(8), aligned(sizeof(OUT))));
    v8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (OUT)acc[e];
    if (STREAM) __builtin_nontemporal_store(o, reinterpret_cast<v8*>(yp));
    else *reinterpret_cast<v8*>(yp) = o;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < N - n) yp[e] = (OUT)acc[e];
  }
}

// Threads of a row, in how many workgroups of how many threads.
struct RowGroups {
  int64_t per_row, parts, threads;
};
RowGroups row_groups(int64_t N) {
  const int64_t per_row = (N + 7) / 8, parts = (per_row + 1023) / 1024;
  return {per_row, parts, ((per_row + parts - 1) / parts + 63) / 64 * 64};
}

template <typename T, typename OUT>
int launch_combine(const void* x, const float* weights, const int32_t* slots, const void* add, void* y, int R, int M,
                   int top, int N, hipStream_t st) {
  const RowGroups g = row_groups(N);
  const T* xp = static_cast<const T*>(x);
  const OUT* ap = static_cast<const OUT*>(add);
  OUT* yp = static_cast<OUT*>(y);
  const bool stream = (int64_t)M * top * N * (int64_t)sizeof(T) >= kCacheBytes;
  if (g.per_row >= 64 && stream)
    combine_kernel<T, OUT, true, true><<<(unsigned)(M * g.parts), (unsigned)g.threads, 0, st>>>(
        xp, weights, slots, ap, yp, R, M, top, N, (uint32_t)g.per_row, (uint32_t)g.parts);
  else if (g.per_row >= 64)
    combine_kernel<T, OUT, true, false><<<(unsigned)(M * g.parts), (unsigned)g.threads, 0, st>>>(
        xp, weights, slots, ap, yp, R, M, top, N, (uint32_t)g.per_row, (uint32_t)g.parts);
  else
    combine_kernel<T, OUT, false, false><<<(unsigned)((M * g.per_row + 255) / 256), 256, 0, st>>>(
        xp, weights, slots, ap, yp, R, M, top, N, (uint32_t)g.per_row, 1);
  return launch_status();
}

}  // namespace

int64_t route_experts_bytes(int64_t M, int64_t E) {
  const int64_t chunks = chunks_of(M);
  return chunks <= 1 ? 0 : chunks * pitch_of((int)E) * (int64_t)sizeof(uint16_t);
}

int launch_route_experts(const void* logits, int type, int64_t ld, const float* bias, int score, int renormalize,
                         float scale, int top, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                         int32_t* slots, void* workspace, int M, int E, hipStream_t st) {
  const Route a{logits, ld, bias, score, renormalize, scale, top, ids, weights, offsets, rows, slots,
                static_cast<uint16_t*>(workspace), M, E, passes_of(M)};
  if (type == PRISM_TYPE_F32) return launch_bias<float>(a, st);
  if (type == PRISM_TYPE_F16) return launch_bias<_Float16>(a, st);
  return launch_bias<__bf16>(a, st);
}

int64_t combine_threads(int64_t M, int64_t N) {
  const RowGroups g = row_groups(N);
  return g.per_row >= 64 ? M * g.parts * g.threads : (M * g.per_row + 255) / 256 * 256;
}

int launch_combine_experts(const void* x, int type, const float* weights, const int32_t* slots, const void* add,
                           void* y, int y_type, int R, int M, int top, int N, hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch_combine<float, float>(x, weights, slots, add, y, R, M, top, N, st);
  if (type == PRISM_TYPE_F16) {
    if (y_type == type) return launch_combine<_Float16, _Float16>(x, weights, slots, add, y, R, M, top, N, st);
    return launch_combine<_Float16, float>(x, weights, slots, add, y, R, M, top, N, st);
  }
  if (y_type == type) return launch_combine<__bf16, __bf16>(x, weights, slots, add, y, R, M, top, N, st);
  return launch_combine<__bf16, float>(x, weights, slots, add, y, R, M, top, N, st);
}

}  // namespace prism
