// fp8 (e4m3) quantizers of the block-128 linear layer: activations in 1 x 128
// blocks, weights in 128 x 128 tiles, and SwiGLU with the activation
// quantizer behind it.  The method's pages quantize activations to 8 bits
// ahead of each product (StartLux-Prism README, "Quick start"); these are the
// 8-bit floating point counterparts of prism_quantize_rows.
//
// All three read each value once with 16-byte loads, keep it in registers
// between the absmax and the codes, and write each code once: they are bound
// by HBM.  16 neighbouring lanes hold one 128-block, 8 values each, so the
// absmax of a block is four cross-lane steps and no LDS.  Kernels alone against
// a large copy's rate: 8192 x 5120 bf16 25.0 us (floor 25), tiles of 17400 x 5120
// bf16 56.6 us (53), SwiGLU of 2048 x 17360 bf16 37.1 us (35); 16 x 5120 fp32 and
// SwiGLU of 4 x 9728, 2.8 us each, are the latency of one load, one reduction and
// one store.  Back to back, with the writes of the call before still under way,
// the large ones take 28, 55 and 40 us.
#include "fp8_math.h"

namespace prism {
namespace {

using namespace fp8;

__device__ inline uint32_t max16(uint32_t m) {
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  return m;
}

// h = g / (1 + exp(-g)) * u as (1 / (1 / 16 + exp(-g) / 16) / 16) * g * u: the
// reciprocal is v_rcp_f32 (1 ulp), and the 16 keeps it a normal number down to
// g = -90; below it is 0.  It is scaled back before g is multiplied in, so that
// a subnormal gate keeps its bits.  exp's argument is one fma with the rounding
// of fp32, |g| 2^-24 relative (5e-6 at g = -80).  All of it is four orders
// below a code's half step, and an IEEE division would be a third of the
// kernel's instructions (2048 x 17360 bf16: 42.3 us).
__device__ inline float swiglu(float g, float u) {
  const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(g, -0x1.715476p+0f, -4.0f));
  return __builtin_amdgcn_rcpf(e + 0x1p-4f) * 0x1p-4f * g * u;
}

// One 16-lane group per 1 x 128 block and step; a workgroup takes 16 rows by
// U consecutive blocks.  GLU: x holds the gates, up the factors.
template <typename T, int U, bool GLU>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const T* __restrict__ x, const T* __restrict__ up,
                                                              int64_t ld, uint8_t* __restrict__ q,
                                                              float* __restrict__ scale, int64_t M, int K,
                                                              int col_groups) {
  const int64_t row = (int64_t)(blockIdx.x / (unsigned)col_groups) * 16 + (threadIdx.x >> 4);
  const int b0 = (int)(blockIdx.x % (unsigned)col_groups) * U;
  const int li = threadIdx.x & 15;
  if (row >= M) return;  // whole 16-lane groups leave together
  float v[U][8];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int k = (b0 + i) * kBlock + li * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    if (k < K) {  // K is a multiple of 16: eight values are inside or outside together
      load8(x + row * ld + k, v[i]);
      if constexpr (GLU) {
        float u[8];
        load8(up + row * ld + k, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = swiglu(v[i][e], u[e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int k = (b0 + i) * kBlock + li * 8;
    const float s = block_scale(max16(absmax8(v[i])));
    if (li == 0 && k < K) scale[(int64_t)(b0 + i) * M + row] = s;
    if (k < K) *reinterpret_cast<v2i*>(q + row * K + k) = codes8(v[i], s);
  }
}

// One workgroup per 128 x 128 tile: 16 rows per step, 8 steps, all values in
// registers while the tile's absmax is joined through LDS.
template <typename T>
__global__ __launch_bounds__(256) void quantize_tiles_kernel(const T* __restrict__ x, int64_t ld,
                                                             uint8_t* __restrict__ q, float* __restrict__ scale,
                                                             int64_t M, int K, int kb) {
  __shared__ uint32_t part[4];
  const int64_t tr = blockIdx.x / (unsigned)kb;
  const int b = (int)(blockIdx.x % (unsigned)kb);
  const int k = b * kBlock + (threadIdx.x & 15) * 8;
  const int64_t row0 = tr * kBlock + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    if (k < K && row0 + 16 * i < M) load8(x + (row0 + 16 * i) * ld + k, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, absmax8(v[i]));
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const float s = block_scale(m);
  if (threadIdx.x == 0) scale[tr * kb + b] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k < K && row0 + 16 * i < M) *reinterpret_cast<v2i*>(q + (row0 + 16 * i) * K + k) = codes8(v[i], s);
}

// Blocks per lane group: two once there are many workgroups per CU, since
// fewer cache lines are then shared by workgroups of different dies where rows
// do not start on a line (2048 x 17360 SwiGLU 38.8 -> 36.8 us; 8192 x 5120 26.4
// -> 24.9; one block is faster below, 2048 x 2560 5.5 against 5.7).
int blocks_per_group(int64_t M, int64_t K) { return (M + 15) / 16 * ((K + kBlock - 1) / kBlock) >= 4096 ? 2 : 1; }

template <typename T, bool GLU>
int launch_blocks(const void* x, const void* up, int64_t ld, uint8_t* q, float* scale, int64_t M, int64_t K,
                  hipStream_t st) {
  const T* xp = static_cast<const T*>(x);
  const T* upp = static_cast<const T*>(up);
  const unsigned groups = (unsigned)quantize_blocks_groups(M, K);
  const int cg = (int)(groups / ((M + 15) / 16));
  if (blocks_per_group(M, K) == 2)
    quantize_blocks_kernel<T, 2, GLU><<<groups, 256, 0, st>>>(xp, upp, ld, q, scale, M, (int)K, cg);
  else
    quantize_blocks_kernel<T, 1, GLU><<<groups, 256, 0, st>>>(xp, upp, ld, q, scale, M, (int)K, cg);
  return launch_status();
}

template <typename T>
int launch_tiles(const void* x, int64_t ld, uint8_t* q, float* scale, int64_t M, int64_t K, hipStream_t st) {
  const int kb = (int)((K + kBlock - 1) / kBlock);
  quantize_tiles_kernel<T><<<(unsigned)quantize_tiles_groups(M, K), 256, 0, st>>>(static_cast<const T*>(x), ld, q, scale, M, (int)K, kb);
  return launch_status();
}

}  // namespace

int64_t quantize_blocks_groups(int64_t M, int64_t K) {
  const int64_t kb = (K + kBlock - 1) / kBlock, per = blocks_per_group(M, K);
  return (M + 15) / 16 * ((kb + per - 1) / per);
}

int64_t quantize_tiles_groups(int64_t N, int64_t K) {
  return (N + kBlock - 1) / kBlock * ((K + kBlock - 1) / kBlock);
}

int launch_quantize_blocks_fp8(const void* x, int type, int64_t ld, uint8_t* q, float* scale, int64_t M, int64_t K,
                               hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch_blocks<float, false>(x, nullptr, ld, q, scale, M, K, st);
  if (type == PRISM_TYPE_F16) return launch_blocks<_Float16, false>(x, nullptr, ld, q, scale, M, K, st);
  return launch_blocks<__bf16, false>(x, nullptr, ld, q, scale, M, K, st);
}

int launch_swiglu_quantize_fp8(const void* gate, const void* up, int type, int64_t ld, uint8_t* q, float* scale,
                               int64_t M, int64_t K, hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch_blocks<float, true>(gate, up, ld, q, scale, M, K, st);
  if (type == PRISM_TYPE_F16) return launch_blocks<_Float16, true>(gate, up, ld, q, scale, M, K, st);
  return launch_blocks<__bf16, true>(gate, up, ld, q, scale, M, K, st);
}

int launch_quantize_tiles_fp8(const void* x, int type, int64_t ld, uint8_t* q, float* scale, int64_t M, int64_t K,
                              hipStream_t st) {
  if (type == PRISM_TYPE_F32) return launch_tiles<float>(x, ld, q, scale, M, K, st);
  if (type == PRISM_TYPE_F16) return launch_tiles<_Float16>(x, ld, q, scale, M, K, st);
  return launch_tiles<__bf16>(x, ld, q, scale, M, K, st);
}

}  // namespace prism
