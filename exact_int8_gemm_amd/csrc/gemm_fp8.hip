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
// its products to their largest before it adds them: measured on MI355X
// against 64-bit sums, its error reaches 2^-10.9 of the largest product of the
// block (2-norm over N(0, 1) operands: 1.4e-5; with one activation per block
// 50 times the others: 3.8e-5).  That is below the rounding of a 16-bit y
// (bf16 1.7e-3, f16 2.1e-4) and of the codes themselves (2^-4), but not what
// an fp32 y promises.  So 16-bit outputs take that instruction, and an fp32 y
// takes four v_mfma_f32_16x16x32_f16 on the codes converted to f16 in
// registers: every e4m3 value and product is exact there, and the error is
// that of fp32 sums (2-norm 1e-8), at half the matrix rate.
//
// Lane layout (both): lane l supplies row (A) or column (B) l % 16; its 32
// codes of a block are the two 16-byte chunks l / 16 and l / 16 + 4.  Result
// register r of lane l is row 4 (l / 16) + r, column l % 16.
#include "fp8_math.h"
#include "lds_copy.h"

namespace prism {
namespace {

using tiled::kOutOfRange;
using tiled::make_rsrc;
using fp8::kBlock;

typedef int v8i __attribute__((ext_vector_type(8)));

// 32 codes of a lane: chunk l / 16 and chunk l / 16 + 4 of a 128-block.
struct Frag {
  v4i lo, hi;
};

template <bool EXACT>
struct Operand;

template <>
struct Operand<false> {
  v8i v;
  __device__ inline explicit Operand(const Frag& f)
      : v{f.lo[0], f.lo[1], f.lo[2], f.lo[3], f.hi[0], f.hi[1], f.hi[2], f.hi[3]} {}
};

template <>
struct Operand<true> {
  fp8::v8h v[4];
  __device__ inline explicit Operand(const Frag& f) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t u = (uint32_t)(s < 2 ? f.lo[2 * s + h] : f.hi[2 * (s - 2) + h]);
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, true);
        v[s][4 * h] = a[0];
        v[s][4 * h + 1] = a[1];
        v[s][4 * h + 2] = b[0];
        v[s][4 * h + 3] = b[1];
      }
    }
  }
};

__device__ inline v4f block_sum(const Operand<false>& a, const Operand<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ inline v4f block_sum(const Operand<true>& a, const Operand<true>& b) {
  v4f p{0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[s], b.v[s], p, 0, 0, 0);
  return p;
}

// One wave per 16 x 16 output tile, operands straight from global memory.
template <typename OUT, bool EXACT>
__global__ __launch_bounds__(256) void gemm_fp8_wave_kernel(const uint8_t* __restrict__ q,
                                                            const float* __restrict__ s_a,
                                                            const uint8_t* __restrict__ w,
                                                            const float* __restrict__ s_w, OUT* __restrict__ y, int M,
                                                            int N, int K, int tiles_n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)tiles_n) * 16;
  const int64_t n0 = ((int64_t)(blockIdx.x % (unsigned)tiles_n) * 4 + wave) * 16;
  if (n0 >= N) return;
  const int KB = (K + kBlock - 1) / kBlock;
  const auto ra = make_rsrc(q + m0 * K, (M - m0) * K);
  const auto rb = make_rsrc(w + n0 * K, (N - n0) * K);
  auto load = [&](__amdgpu_buffer_rsrc_t rs, bool in, int b) {
    Frag f;
    const int k0 = b * kBlock + 16 * g, k1 = k0 + 64;
    f.lo = __builtin_amdgcn_raw_buffer_load_b128(rs, in && k0 < K ? (uint32_t)(r * K + k0) : kOutOfRange, 0, 0);
    f.hi = __builtin_amdgcn_raw_buffer_load_b128(rs, in && k1 < K ? (uint32_t)(r * K + k1) : kOutOfRange, 0, 0);
    return f;
  };
  v4f f{0, 0, 0, 0};
  for (int b = 0; b < KB; ++b) {
    const Operand<EXACT> a(load(ra, m0 + r < M, b)), c(load(rb, n0 + r < N, b));
    const v4f p = block_sum(a, c);
    const float sw = s_w[(n0 / kBlock) * KB + b];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 4 * g + i;
      const float sa = m < M ? s_a[(int64_t)b * M + m] : 0.0f;
      f[i] = __builtin_fmaf(p[i], sa * sw, f[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + 4 * g + i;
    if (m < M && n0 + r < N) y[m * N + n0 + r] = (OUT)f[i];
  }
}

template <typename OUT, bool EXACT>
int launch(const uint8_t* q, const float* s_a, const uint8_t* w, const float* s_w, void* y, int M, int N, int K,
           hipStream_t st) {
  const int tiles_n = (N + 63) / 64;
  const int64_t grid = (int64_t)((M + 15) / 16) * tiles_n;
  gemm_fp8_wave_kernel<OUT, EXACT>
      <<<(unsigned)grid, 256, 0, st>>>(q, s_a, w, s_w, static_cast<OUT*>(y), M, N, K, tiles_n);
  return launch_status();
}

}  // namespace

int launch_gemm_fp8(const uint8_t* q, const float* s_a, const uint8_t* w, const float* s_w, void* y, int type, int M,
                    int N, int K, hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch<float, true>(q, s_a, w, s_w, y, M, N, K, st);
  if (type == PRISM_TYPE_F16) return launch<_Float16, false>(q, s_a, w, s_w, y, M, N, K, st);
  return launch<__bf16, false>(q, s_a, w, s_w, y, M, N, K, st);
}

}  // namespace prism
