// reduce_kernels.cuh -- the second half of a product whose k-ranges were
// summed separately (kEpiPartial of fused_kernel.cuh): adds the fp32 partials
// in k order, so results do not depend on timing, and applies the epilogue.
// Bound by the partials' bytes, which sit in L2 (the rows are few).
#pragma once
#include "act.cuh"
#include "ptx_ops.cuh"

namespace gb300 {
namespace ops {

enum ReduceMode : int { kReduceStore = 0, kReduceGlu = 1, kReduceGluBwd = 2 };

struct ReduceArgs {
  const float* partial;  // [split][M][ld], `stride` floats from one split to the next
  int64_t ld, stride;
  int32_t splits, M, N;  // N: columns of the output (h's for the gated modes)
  int32_t bf16, act;
  uint16_t* out;         // kReduceStore: [M, N]; gated modes: h [M, N] (rows ld_out apart)
  int64_t ld_out;
  uint16_t* gu;          // kReduceGlu: written unless null; kReduceGluBwd: read; [M, 2N]
  uint16_t* dgu;         // kReduceGluBwd: [M, 2N]
};

// Four neighbouring columns per thread (N is a multiple of 8).
template <int kMode>
__global__ void __launch_bounds__(256) reduce_kernel(const ReduceArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t cols4 = a.N / 4;
  const int64_t total = cols4 * a.M;
  const bool bf16 = a.bf16 != 0;
  auto sum = [&](const float* p) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int32_t k = 0; k < a.splits; ++k) {
      const float4 v = ptx::ld_global_cg_v4(p + k * a.stride);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    return s;
  };
  auto store4 = [&](uint16_t* p, float x, float y, float z, float w) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack16(bf16, x, y), pack16(bf16, z, w));
  };
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t m = i / cols4, n = (i - m * cols4) * 4;
    const float* p = a.partial + m * a.ld + n;
    const float4 s = sum(p);
    if constexpr (kMode == kReduceStore) {
      store4(a.out + m * a.ld_out + n, s.x, s.y, s.z, s.w);
    } else if constexpr (kMode == kReduceGlu) {
      const float4 u = sum(p + a.N);
      store4(a.out + m * a.ld_out + n, act_value(a.act, s.x) * u.x, act_value(a.act, s.y) * u.y,
             act_value(a.act, s.z) * u.z, act_value(a.act, s.w) * u.w);
      if (a.gu) {
        store4(a.gu + m * 2 * a.N + n, s.x, s.y, s.z, s.w);
        store4(a.gu + m * 2 * a.N + a.N + n, u.x, u.y, u.z, u.w);
      }
    } else {
      const uint2 gw = *reinterpret_cast<const uint2*>(a.gu + m * 2 * a.N + n);
      const uint2 uw = *reinterpret_cast<const uint2*>(a.gu + m * 2 * a.N + a.N + n);
      const float2 g0 = unpack16(bf16, gw.x), g1 = unpack16(bf16, gw.y);
      const float2 u0 = unpack16(bf16, uw.x), u1 = unpack16(bf16, uw.y);
      float av[4], sv[4];
      act_both(a.act, g0.x, av[0], sv[0]);
      act_both(a.act, g0.y, av[1], sv[1]);
      act_both(a.act, g1.x, av[2], sv[2]);
      act_both(a.act, g1.y, av[3], sv[3]);
      store4(a.dgu + m * 2 * a.N + n, s.x * u0.x * sv[0], s.y * u0.y * sv[1], s.z * u1.x * sv[2],
             s.w * u1.y * sv[3]);
      store4(a.dgu + m * 2 * a.N + a.N + n, s.x * av[0], s.y * av[1], s.z * av[2], s.w * av[3]);
      store4(a.out + m * a.ld_out + n, av[0] * u0.x, av[1] * u0.y, av[2] * u1.x, av[3] * u1.y);
    }
  }
}

}  // namespace ops
}  // namespace gb300
