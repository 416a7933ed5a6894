// norm_kernels.cuh -- layer norm and RMS norm of rows, and their gradients.
//
//   layer norm  m = mean x, v = mean (x - m)^2, r = 1 / sqrt(v + eps), h = (x - m) r
//   RMS norm    r = 1 / sqrt(mean x^2 + eps), h = x r
//   y = h w (+ b)
// and from dy, with q = dy w:
//   dx = r (q - mean q - h mean(q h))        (RMS norm: without mean q)
//   dw = sum over the rows of dy h,  db = sum over the rows of dy
//
// Sums and statistics are fp32.  The mean is taken twice: the second pass sums
// d = x - m1 and d^2 about the first pass's m1, whose rounding (2^-24 m1, which
// a row far from zero shows) c = mean d takes back: m = m1 + c, v = mean d^2 - c^2.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx_ops.cuh"

namespace gb300 {
namespace ops {

struct NormArgs {
  const void *x, *dy, *weight, *bias;  // weight, bias: null for 1 and 0
  void* y;                             // y, or dx
  float* stats;                        // [T][2]: m, r; RMS norm [T][1]: r; null: not kept
  int64_t ldx, lddy, ldy, T, D;
  float eps;
  float* partial;  // [chunks][2][D]: sums of dy h and of dy over a chunk's rows
  int64_t chunks;
  void *dweight, *dbias;  // null: not wanted
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float* p) { *p = v; }
__device__ __forceinline__ void narrow(float v, __half* p) { *p = __float2half_rn(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// Sums of a and b over the block, the same in every thread; the order is fixed.
// sm: 64 floats, free again after the next barrier.
__device__ __forceinline__ float2 block_sums(float a, float b, float* sm) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    sm[threadIdx.x >> 5] = a;
    sm[32 + (threadIdx.x >> 5)] = b;
  }
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < warps; ++i) s.x += sm[i], s.y += sm[32 + i];
  __syncthreads();
  return s;
}

// One block per row, element by element: rows of any length, start and distance.
template <class X, class W, bool kRms>
__global__ void __launch_bounds__(512) norm_any(const NormArgs a) {
  __shared__ float sm[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + t * a.ldx;
  X* y = static_cast<X*>(a.y) + t * a.ldy;
  const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
  const float n = static_cast<float>(a.D);
  float m1 = 0.0f;
  if (!kRms) {
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) s += widen(x[i]);
    m1 = block_sums(s, 0.0f, sm).x / n;
  }
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    const float d = widen(x[i]) - m1;
    s1 += d;
    s2 = fmaf(d, d, s2);
  }
  const float2 s = block_sums(s1, s2, sm);
  const float c = kRms ? 0.0f : s.x / n;
  const float v = s.y / n - c * c;
  const float r = __frsqrt_rn((v < 0.0f ? 0.0f : v) + a.eps);  // (fmaxf would lose a NaN)
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    float v = ((widen(x[i]) - m1) - c) * r;
    if (w) v *= widen(w[i]);
    if (b) v += widen(b[i]);
    narrow(v, y + i);
  }
  if (a.stats && threadIdx.x == 0) {
    if (kRms) {
      a.stats[t] = r;
    } else {
      a.stats[2 * t] = m1 + c;
      a.stats[2 * t + 1] = r;
    }
  }
}

template <class X, class W, bool kRms>
__global__ void __launch_bounds__(512) norm_dx_any(const NormArgs a) {
  __shared__ float sm[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const X *x = static_cast<const X*>(a.x) + t * a.ldx, *dy = static_cast<const X*>(a.dy) + t * a.lddy;
  X* dx = static_cast<X*>(a.y) + t * a.ldy;
  const W* w = static_cast<const W*>(a.weight);
  const float n = static_cast<float>(a.D);
  const float m = kRms ? 0.0f : a.stats[2 * t], r = kRms ? a.stats[t] : a.stats[2 * t + 1];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    const float h = (widen(x[i]) - m) * r, q = widen(dy[i]) * (w ? widen(w[i]) : 1.0f);
    s1 += q;
    s2 = fmaf(q, h, s2);
  }
  const float2 s = block_sums(s1, s2, sm);
  const float c1 = kRms ? 0.0f : s.x / n, c2 = s.y / n;
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    const float h = (widen(x[i]) - m) * r, q = widen(dy[i]) * (w ? widen(w[i]) : 1.0f);
    narrow(r * ((q - c1) - h * c2), dx + i);
  }
}

// grid (columns / 32, chunks), block 32 x 8: sums of dy h and dy over a chunk.
template <class X, bool kRms>
__global__ void __launch_bounds__(256) norm_dw_any(const NormArgs a) {
  __shared__ float sm[2][8][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t t0 = blockIdx.y * a.T / a.chunks, t1 = (blockIdx.y + 1) * a.T / a.chunks;
  const X *x = static_cast<const X*>(a.x) + col, *dy = static_cast<const X*>(a.dy) + col;
  float sw = 0.0f, sb = 0.0f;
  if (col < a.D)
    for (int64_t t = t0 + warp; t < t1; t += 8) {
      const float m = kRms ? 0.0f : a.stats[2 * t], r = kRms ? a.stats[t] : a.stats[2 * t + 1];
      const float g = widen(dy[t * a.lddy]);
      sw = fmaf(g, (widen(x[t * a.ldx]) - m) * r, sw);
      sb += g;
    }
  sm[0][warp][lane] = sw;
  sm[1][warp][lane] = sb;
  __syncthreads();
  if (warp < 2 && col < a.D) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[warp][i][lane];
    a.partial[(2 * static_cast<int64_t>(blockIdx.y) + warp) * a.D + col] = s;
  }
}

// The sums of all chunks, in order: thread (column, weight or bias).
template <class W>
__global__ void __launch_bounds__(256) norm_dw_sum(const NormArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  W* out = static_cast<W*>(blockIdx.y == 0 ? a.dweight : a.dbias);
  if (col >= a.D || !out) return;
  float s = 0.0f;
  for (int64_t c = 0; c < a.chunks; ++c) s += a.partial[(2 * c + blockIdx.y) * a.D + col];
  narrow(s, out + col);
}

}  // namespace ops
}  // namespace gb300
