// ortho_kernels.cuh -- the memory-bound ends of the orthogonalised update:
// the sum of squares of each matrix, its scaled split into a high and a low
// fp16 part, and the sum of the two parts in the output's type.  Bound by their
// bytes, or by a launch where they are few (4096 x 8192 from and to fp32 and
// fp16: 3 launches of 15 to 40 us beside 4900 us of products; 512 x 512: 3 to 5
// us each).  A single kernel for norm and split would have to wait for all
// blocks in between; a launch does that for less.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "act.cuh"
#include "ptx_ops.cuh"

namespace gb300 {
namespace ops {

enum DType : int32_t { kF16 = 0, kBF16 = 1, kF32 = 2 };

constexpr int kNormBlocks = 128;  // partial sums per matrix

struct OrthoArgs {
  const void* in;       // [batch][rows][cols], rows ld apart, matrices bs apart
  int64_t ld, bs;
  int32_t dtype;
  int32_t rows, cols;
  uint16_t* x;          // [batch][2][rows][pitch]
  int64_t pitch;
  float* partial;       // [batch][kNormBlocks]
  float eps, scale;     // scale: X is held as scale X
  void* out;            // ortho_join: [batch][rows][cols]
  int64_t ld_out, bs_out;
};

__device__ __forceinline__ float load_any(int32_t dtype, const void* p, int64_t i) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  return widen16(dtype == kBF16, static_cast<const uint16_t*>(p)[i]);
}

// Sum over the block, the same in every thread; the order is fixed.
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) s += sm[i];
  return s;
}

// grid (kNormBlocks, batch): partial sums of squares.
__global__ void __launch_bounds__(256) ortho_norm(const OrthoArgs a) {
  __shared__ float sm[8];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t base = blockIdx.y * a.bs;
  float s = 0.0f;
  for (int32_t r = blockIdx.x; r < a.rows; r += gridDim.x)
    for (int32_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float v = load_any(a.dtype, a.in, base + r * a.ld + c);
      s = fmaf(v, v, s);
    }
  s = block_sum(s, sm);
  if (threadIdx.x == 0) a.partial[blockIdx.y * kNormBlocks + blockIdx.x] = s;
}

// grid (blocks, batch): X = scale in / (|in| + eps), as high + low.
__global__ void __launch_bounds__(256) ortho_split(const OrthoArgs a) {
  __shared__ float sm[8];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const float p = threadIdx.x < kNormBlocks ? a.partial[blockIdx.y * kNormBlocks + threadIdx.x] : 0.0f;
  const float f = a.scale / (sqrtf(block_sum(p, sm)) + a.eps);
  const int64_t base = blockIdx.y * a.bs;
  const int64_t part = a.rows * a.pitch;
  uint16_t* x = a.x + blockIdx.y * 2 * part;
  for (int32_t r = blockIdx.x; r < a.rows; r += gridDim.x)
    for (int32_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float v = f * load_any(a.dtype, a.in, base + r * a.ld + c);
      const __half h = __float2half_rn(v);
      const __half l = __float2half_rn(v - __half2float(h));
      x[r * a.pitch + c] = *reinterpret_cast<const uint16_t*>(&h);
      x[part + r * a.pitch + c] = *reinterpret_cast<const uint16_t*>(&l);
    }
}

// grid (blocks, batch): out = (high + low) / scale.
__global__ void __launch_bounds__(256) ortho_join(const OrthoArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t part = a.rows * a.pitch;
  const uint16_t* x = a.x + blockIdx.y * 2 * part;
  const float f = 1.0f / a.scale;
  for (int32_t r = blockIdx.x; r < a.rows; r += gridDim.x)
    for (int32_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float v = f * (widen16(false, x[r * a.pitch + c]) + widen16(false, x[part + r * a.pitch + c]));
      const int64_t i = blockIdx.y * a.bs_out + r * a.ld_out + c;
      if (a.dtype == kF32)
        static_cast<float*>(a.out)[i] = v;
      else
        static_cast<uint16_t*>(a.out)[i] = round16(a.dtype == kBF16, v);
    }
}

}  // namespace ops
}  // namespace gb300
