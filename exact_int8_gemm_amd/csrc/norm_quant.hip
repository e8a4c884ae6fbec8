// Root-mean-square norm with the residual's addition in front of it and an 8-bit
// quantizer behind it, in one pass: what stands in front of each quantized
// product of a layer (the method's pages quantize activations to 8 bits ahead
// of each product; StartLux-Prism README, "Quick start").
//
//   h = x + residual, rounded to the residual's type (h = x without one)
//   inv = 1 / sqrt(sum h^2 / K + eps), rounded once to fp32
//   y = (h inv) gain, each product rounded to fp32
// and the codes and scales of y: e4m3 with a scale per 128 values, or int8 with a
// scale per row, whose scale is one product with 1 / 127.
//
// The sum of squares is held in 64 bits: each square is exact there, and what
// the order of the sum changes is 2^-53 of it, below the rounding to fp32 but
// for one row in 10^8.  The order depends on K alone all the same, so a row has the
// same bits in any batch.
//
// One workgroup per row.  The row is read once with 16-byte loads and stays in
// registers, eight values in each of a thread's C chunks.  Bound by HBM: 8192 x 5120
// bf16 with an fp32 residual to int8, 461 MB, 81 us (5.7 TB/s; a large copy makes
// 5.1); 1999 x 9680 fp16 with the norm itself, 174 MB, 34 us; one row of 5120, 3.9 us,
// is two reductions one behind the other.  The scattered stores of the fp8 scales, 4
// bytes in a line of their own each, are 4% of it.
#include "fp8_math.h"
#include "quant_math.h"

namespace prism {
namespace {

using namespace fp8;

// Eight values of a PRISM_TYPE_* from element `at`.
__device__ inline void load8_of(const void* p, int type, int64_t at, float* x) {
  if (type == PRISM_TYPE_F32) load8(static_cast<const float*>(p) + at, x);
  else if (type == PRISM_TYPE_F16) load8(static_cast<const _Float16*>(p) + at, x);
  else load8(static_cast<const __bf16*>(p) + at, x);
}

template <bool PAST, typename T>
__device__ inline void store8(T* p, const float* x) {
  typedef T v8 __attribute__((ext_vector_type(8)));
  v8 o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = (T)x[e];
  if (PAST) __builtin_nontemporal_store(o, reinterpret_cast<v8*>(p));
  else *reinterpret_cast<v8*>(p) = o;
}

constexpr int kMaxWaves = 16;

struct Norm {
  const void* x;
  int64_t x_ld;
  const void* residual;
  int64_t res_ld;
  void* residual_out;
  int64_t out_ld;
  const void* gain;
  int gain_type;
  double eps;
  void* norm;
  void* q;
  float* scale;
  int64_t M;
  int K;
};

// A residual of this many bytes is written past the caches: it is read again behind a whole part of the
// layer, whose weights alone are more than the caches hold (8192 x 5120, us: fp32
// residual, 168 MB, 80.5, through them 84.7; bf16, 84 MB, 54 both ways; nothing in
// between was measured).
constexpr int64_t kPastBytes = (int64_t)128 << 20;

// T: x's type and norm's; TR: the residual's, PAST: it is written past the caches.
template <typename T, typename TR, bool RES, bool PAST, bool INT8, int C>
__global__ __launch_bounds__(C == 1 ? 512 : 1024) void norm_kernel(const Norm a) {
  __shared__ double sums[kMaxWaves];
  __shared__ uint32_t peaks[kMaxWaves];
  const int64_t row = blockIdx.x;
  const int threads = (int)blockDim.x, waves = threads / 64, wave = (int)threadIdx.x / 64;
  const T* xp = static_cast<const T*>(a.x) + row * a.x_ld;
  float v[C][8];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int k = ((int)threadIdx.x + threads * i) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    if (k >= a.K) continue;
    load8(xp + k, v[i]);
    if constexpr (RES) {
      float r[8];
      load8(static_cast<const TR*>(a.residual) + row * a.res_ld + k, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = (float)(TR)(v[i][e] + r[e]);
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int k = ((int)threadIdx.x + threads * i) * 8;
    if constexpr (RES) {
      if (a.residual_out && k < a.K) store8<PAST>(static_cast<TR*>(a.residual_out) + row * a.out_ld + k, v[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)v[i][e], (double)v[i][e], sum);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((threadIdx.x & 63) == 0) sums[wave] = sum;
  __syncthreads();
  sum = sums[0];
  for (int w = 1; w < waves; ++w) sum += sums[w];
  const float inv = (float)(1.0 / __builtin_sqrt(sum / (double)a.K + a.eps));

#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int k = ((int)threadIdx.x + threads * i) * 8;
    if (k >= a.K) continue;
    float g[8];
    load8_of(a.gain, a.gain_type, k, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * inv * g[e];
    if (a.norm) store8<false>(static_cast<T*>(a.norm) + row * a.K + k, v[i]);
  }
  if constexpr (INT8) {
    uint32_t peak = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) peak = max(peak, absmax8(v[i]));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) peak = max(peak, (uint32_t)__shfl_xor((int)peak, off, 64));
    if ((threadIdx.x & 63) == 0) peaks[wave] = peak;
    __syncthreads();
    peak = peaks[0];
    for (int w = 1; w < waves; ++w) peak = max(peak, peaks[w]);
    const bool finite = peak < 0x7f800000u;
    const float s = finite ? __builtin_bit_cast(float, peak) * (1.0f / 127.0f) : __builtin_nanf("");
    const bool zero = !finite || s == 0.0f;
    const float r = zero ? 0.0f : quant::fast_recip(s);
    if (threadIdx.x == 0) a.scale[row] = s;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int k = ((int)threadIdx.x + threads * i) * 8;
      if (k >= a.K) continue;
      v2i c{0, 0};
      if (!zero) {
        c[0] = (int)quant::pack4(float4{v[i][0], v[i][1], v[i][2], v[i][3]}, s, r);
        c[1] = (int)quant::pack4(float4{v[i][4], v[i][5], v[i][6], v[i][7]}, s, r);
      }
      *reinterpret_cast<v2i*>(static_cast<int8_t*>(a.q) + row * a.K + k) = c;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int chunk = (int)threadIdx.x + threads * i, k = chunk * 8;
      uint32_t peak = absmax8(v[i]);
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) peak = max(peak, (uint32_t)__shfl_xor((int)peak, off, 64));
      if (k >= a.K) continue;
      const float s = block_scale(peak);
      if (chunk % 16 == 0) a.scale[(int64_t)(chunk / 16) * a.M + row] = s;
      *reinterpret_cast<v2i*>(static_cast<uint8_t*>(a.q) + row * a.K + k) = codes8(v[i], s);
    }
  }
}

// Chunks of a thread: one up to 512 threads, two up to 1024 (1999 x 9680 fp16: 33.9
// us, four of 320 threads 36.8), eight for the longest rows.
constexpr int threads_of(int64_t K, int chunks) { return (int)((K / 8 + 64 * chunks - 1) / (64 * chunks) * 64); }
constexpr int chunks_of(int64_t K) { return threads_of(K, 1) <= 512 ? 1 : threads_of(K, 2) <= 1024 ? 2 : 8; }
static_assert(threads_of(PRISM_NORM_K_MAX, 8) <= 1024, "the longest row");

template <typename T, typename TR, bool RES, bool PAST, bool INT8>
int launch_chunks(const Norm& a, hipStream_t st) {
#define PRISM_NORM(C) norm_kernel<T, TR, RES, PAST, INT8, C><<<(unsigned)a.M, threads_of(a.K, C), 0, st>>>(a)
  const int chunks = chunks_of(a.K);
  if (chunks == 1) PRISM_NORM(1);
  else if (chunks == 2) PRISM_NORM(2);
  else PRISM_NORM(8);
#undef PRISM_NORM
  return launch_status();
}

template <typename T, bool INT8>
int launch_residual(const Norm& a, int res_type, hipStream_t st) {
  if (!a.residual) return launch_chunks<T, T, false, false, INT8>(a, st);
  const bool past = a.M * a.K * (res_type == PRISM_TYPE_F32 ? 4 : 2) >= kPastBytes;
  if constexpr (!__is_same(T, float)) {
    if (res_type != PRISM_TYPE_F32)
      return past ? launch_chunks<T, T, true, true, INT8>(a, st) : launch_chunks<T, T, true, false, INT8>(a, st);
  }
  return past ? launch_chunks<T, float, true, true, INT8>(a, st) : launch_chunks<T, float, true, false, INT8>(a, st);
}

template <bool INT8>
int launch_type(const Norm& a, int x_type, int res_type, hipStream_t st) {
  if (x_type == PRISM_TYPE_F32) return launch_residual<float, INT8>(a, res_type, st);
  if (x_type == PRISM_TYPE_F16) return launch_residual<_Float16, INT8>(a, res_type, st);
  return launch_residual<__bf16, INT8>(a, res_type, st);
}

}  // namespace

int64_t norm_threads(int64_t M, int64_t K) { return M * threads_of(K, chunks_of(K)); }

int launch_add_rmsnorm_quantize(const void* x, int x_type, int64_t x_ld, const void* residual, int64_t res_ld,
                                void* residual_out, int64_t out_ld, int res_type, const void* gain, int gain_type,
                                double eps, void* norm, void* q, bool int8, float* scale, int64_t M, int64_t K,
                                hipStream_t st) {
  const Norm a{x, x_ld, residual, res_ld, residual_out, out_ld, gain, gain_type, eps, norm, q, scale, M, (int)K};
  return int8 ? launch_type<true>(a, x_type, res_type, st) : launch_type<false>(a, x_type, res_type, st);
}

}  // namespace prism
