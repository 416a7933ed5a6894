// xent_kernels.cuh -- the ends of the vocabulary's loss, around the products of
// fused_kernel.cuh.  For a token with logits z = x W^T
//
//   lse = log sum exp z,  loss = lse - z[target]   (0 where the token is ignored)
//   dz = (dloss + dlse) exp(z - lse) - dloss [column = target]
//   dx = dz W,  dW = dz^T x
//
// Forward: the product's epilogue leaves for each token and each share of a tile's
// columns a maximum m and s = sum exp(z - m), and the target's logit; xent_join
// joins the shares,  (m1, s1) + (m2, s2) = (M, s1 exp(m1 - M) + s2 exp(m2 - M)),
// M = max(m1, m2).  Where m is infinite, s stands for sum exp(z) itself.
//
// Backward: the logits come again, and dz, a piece of the vocabulary at a time, is
// rounded to 16 bits as an operand of the two products.  In fp16 dz of a mean over
// thousands of tokens would be lost below 6e-8, so dz is held times 2^14 / 2^e, 2^e
// the power of two above the largest |dloss| and |dloss + dlse|: below 2^15, and
// off by at most 2^-25, half of fp16's last step, where the largest is 2^13 at least:
// by 2^-38 of it.  The products undo it in fp32.
//
// Tokens without a gradient (ignored ones, a prompt's) take no part: xent_pack copies
// the others' x side by side, and the three products run on those alone.  Where an
// eighth of 4096 tokens is ignored that saves an eighth of 7900 us, for a copy of 12 us.
#pragma once
#include "fused_kernel.cuh"

namespace gb300 {
namespace ops {

struct XentArgs {
  const int64_t* targets;
  int64_t T, V, ignore;
  // Forward: the shares [shares][T] and the targets' logits.
  const float2* shares;
  int64_t num_shares;
  const float* target_z;
  float *loss, *lse;  // forward: lse may be null; backward: lse is read
  // Backward.
  const float *dloss, *dlse;  // dlse may be null
  int64_t dloss_stride, dlse_stride;
  const void* x;
  XentRow* rows;   // of the tokens that have a gradient, in order
  int32_t *live, *order;  // how many, and which
  void* packed;    // their x, [T][D], rows `pitch` apart; zeros up to a whole k-block of 64
  float* scale;    // what the products are to be multiplied by
  float hold;      // dz is held times hold / 2^e
  // The sums of dx, [slices][T][D] to be added up in order, and dx itself.
  const float* sum;
  int64_t slices;
  void* dx;
  int64_t ldx, lddx, pitch, D;
  int32_t bf16;
};

__device__ __forceinline__ float2 lse_join(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), ref = isinf(top) ? 0.0f : top;
  return make_float2(top, fmaf(a.y, ptx::ex2((a.x - ref) * kLog2e), b.y * ptx::ex2((b.x - ref) * kLog2e)));
}

constexpr int kJoinThreads = 512;

// A block joins the shares of `per` tokens (a power of two up to 32): thread at + per
// group every (512 / per)-th share of token `at` from `group` on; then a warp's lanes
// of a token in pairs, and the warps in order.
__global__ void __launch_bounds__(kJoinThreads) xent_join(const XentArgs a, int32_t per) {
  __shared__ float2 sm[kJoinThreads];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int groups = kJoinThreads / per, at = threadIdx.x % per, group = threadIdx.x / per, warp = threadIdx.x / 32;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * per + at;
  float2 v = make_float2(-INFINITY, 0.0f);
  if (t < a.T)
    for (int64_t i = group; i < a.num_shares; i += 4 * groups) {
      float2 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t j = i + k * groups;
        w[k] = j < a.num_shares ? a.shares[j * a.T + t] : make_float2(-INFINITY, 0.0f);
      }
      v = lse_join(v, lse_join(lse_join(w[0], w[1]), lse_join(w[2], w[3])));
    }
  for (int d = 16; d >= per; d >>= 1)
    v = lse_join(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d)));
  if ((threadIdx.x & 31) < per) sm[warp * per + at] = v;
  __syncthreads();
  if (group == 0 && t < a.T) {
    v = sm[at];
    for (int i = 1; i < kJoinThreads / 32; ++i) v = lse_join(v, sm[i * per + at]);
    const float lse = (isinf(v.x) ? 0.0f : v.x) + logf(v.y);
    const int64_t target = a.targets[t];
    // A target outside the vocabulary has no logit: NaN.
    float loss = 0.0f;
    if (target != a.ignore) loss = target >= 0 && target < a.V ? lse - a.target_z[t] : NAN;
    a.loss[t] = loss;
    if (a.lse) a.lse[t] = lse;
  }
}

// x, its rows `pitch` apart: a warp takes pieces of up to 4 x 256 columns.
__global__ void __launch_bounds__(256) xent_copy(const XentArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t pieces = (a.D + 1023) / 1024, all = pieces * a.T;
  for (int64_t i = blockIdx.x * 8 + threadIdx.x / 32; i < all; i += gridDim.x * 8) {
    const int64_t t = i / pieces, c = (i - t * pieces) * 1024 + (threadIdx.x & 31) * 8;
    const uint16_t* from = static_cast<const uint16_t*>(a.x) + t * a.ldx + c;
    uint16_t* to = static_cast<uint16_t*>(a.packed) + t * a.pitch + c;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j * 256 < a.D) v[j] = ptx::ld_global_v4_u32(from + j * 256);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j * 256 < a.D) ptx::st_global_v4(to + j * 256, v[j].x, v[j].y, v[j].z, v[j].w);
  }
}

constexpr int kPackThreads = 512;

// grid: blocks, each for a share of the tokens; every one looks at all of them for the
// power of two above the largest finite |dloss| and |dloss + dlse| and for the number of
// those with a gradient before its own.  dx of the others is zero.
__global__ void __launch_bounds__(kPackThreads) xent_pack(const XentArgs a) {
  constexpr int kWarps = kPackThreads / 32;
  __shared__ float tops[kWarps];
  __shared__ int32_t counts[kWarps], befores[kWarps], place[kPackThreads];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a, b and the target of token t, from loads that wait for none of one another.
  auto row = [&](int64_t t) {
    const int64_t target = a.targets[t];
    const float dloss = a.dloss[t * a.dloss_stride], dlse = a.dlse ? a.dlse[t * a.dlse_stride] : 0.0f;
    XentRow r;
    r.b = target != a.ignore ? dloss : 0.0f;
    r.a = a.dlse ? r.b + dlse : r.b;
    r.target = -1;
    if (target != a.ignore) {
      if (target >= 0 && target < a.V)
        r.target = static_cast<int32_t>(target);
      else
        r.a = NAN;  // as the loss
    }
    r.lse2 = a.lse[t] * kLog2e;
    return r;
  };
  auto has = [](const XentRow& r) { return !(r.a == 0.0f && r.b == 0.0f); };  // (NaN has)
  const int64_t c0 = a.T * blockIdx.x / gridDim.x, c1 = a.T * (blockIdx.x + 1) / gridDim.x;
  XentRow mine = {};  // this block's tokens are on their way while it looks at all
  if (c0 + threadIdx.x < c1) mine = row(c0 + threadIdx.x);
  float top = 0.0f;
  int32_t count = 0, before = 0;
#pragma unroll 2
  for (int64_t t = threadIdx.x; t < a.T; t += kPackThreads) {
    const XentRow r = row(t);
    if (isfinite(r.a)) top = fmaxf(top, fabsf(r.a));
    if (isfinite(r.b)) top = fmaxf(top, fabsf(r.b));
    count += has(r);
    before += has(r) && t < c0;
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  count = __reduce_add_sync(0xffffffffu, count);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) tops[warp] = top, counts[warp] = count, befores[warp] = before;
  __syncthreads();
  top = 0.0f, count = 0, before = 0;
  for (int i = 0; i < kWarps; ++i) top = fmaxf(top, tops[i]), count += counts[i], before += befores[i];
  int e = 0;
  if (top > 0.0f) frexpf(top, &e);
  e = max(-100, min(100, e));  // both factors stay normal
  const float up = ldexpf(a.hold, -e);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  uint16_t *packed = static_cast<uint16_t*>(a.packed), *dx = static_cast<uint16_t*>(a.dx);
  for (int64_t t0 = c0; t0 < c1; t0 += kPackThreads) {
    const int64_t t = t0 + threadIdx.x;
    XentRow r = mine;
    if (t0 > c0 && t < c1) r = row(t);
    const bool own = t < c1 && has(r);
    const uint32_t votes = __ballot_sync(0xffffffffu, own);
    __syncthreads();  // counts and place are read
    if (lane == 0) counts[warp] = __popc(votes);
    __syncthreads();
    int32_t at = before + __popc(votes & ((1u << lane) - 1u));
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) at += counts[i];
      before += counts[i];
    }
    place[threadIdx.x] = own ? at : -1;
    if (own) {
      r.a *= up;
      r.b *= up;
      a.rows[at] = r;
      a.order[at] = static_cast<int32_t>(t);
    }
    __syncthreads();
    // The warps take pieces of up to 4 x 256 columns of the rows in turn.
    const int64_t pieces = (a.D + 1023) / 1024, all = pieces * min(c1 - t0, static_cast<int64_t>(kPackThreads));
    for (int64_t i = warp; i < all; i += kWarps) {
      const int64_t k = i / pieces, c = (i - k * pieces) * 1024 + lane * 8;
      const int32_t to = place[k];
      const uint16_t* from = x + (t0 + k) * a.ldx;
      uint16_t* dst = to >= 0 ? packed + to * a.pitch : dx + (t0 + k) * a.lddx;
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (to >= 0 && c + j * 256 < a.D) v[j] = ptx::ld_global_v4_u32(from + c + j * 256);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j * 256 < a.D) ptx::st_global_v4(dst + c + j * 256, v[j].x, v[j].y, v[j].z, v[j].w);
    }
  }
  if (blockIdx.x + 1 == gridDim.x) {
    const int64_t end = min(a.T, static_cast<int64_t>(max(64, (count + 63) / 64 * 64))) * a.pitch;
    for (int64_t i = count * a.pitch + threadIdx.x * 8; i < end; i += kPackThreads * 8)
      ptx::st_global_v4(packed + i, 0, 0, 0, 0);
    if (threadIdx.x == 0) {
      *a.scale = ldexpf(1.0f / a.hold, e);
      *a.live = count;
    }
  }
}

// dx = scale sum, rounded, to the tokens' own rows: eight columns a thread (D is a
// multiple of 8).
__global__ void __launch_bounds__(256) xent_dx(const XentArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const float scale = *a.scale;
  const bool bf16 = a.bf16 != 0;
  const int64_t per = a.D / 8, n = *a.live * per, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    const int64_t t = i / per, c = (i - t * per) * 8;
    float4 u = make_float4(0, 0, 0, 0), v = u;
#pragma unroll 4
    for (int64_t k = 0; k < a.slices; ++k) {
      const float* p = a.sum + (k * a.T + t) * a.D + c;
      const float4 p0 = ptx::ld_global_cg_v4(p), p1 = ptx::ld_global_cg_v4(p + 4);
      u.x += p0.x, u.y += p0.y, u.z += p0.z, u.w += p0.w;
      v.x += p1.x, v.y += p1.y, v.z += p1.z, v.w += p1.w;
    }
    ptx::st_global_v4(static_cast<uint16_t*>(a.dx) + a.order[t] * a.lddx + c, pack16(bf16, u.x * scale, u.y * scale),
                      pack16(bf16, u.z * scale, u.w * scale), pack16(bf16, v.x * scale, v.y * scale),
                      pack16(bf16, v.z * scale, v.w * scale));
  }
}

}  // namespace ops
}  // namespace gb300
