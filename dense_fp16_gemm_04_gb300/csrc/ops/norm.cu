// norm.cu -- host side of the norms.
#include "norm_host.cuh"

namespace {

using namespace gb300::ops;

// Blocks of a kernel that fit on an SM at once (the SMs of every device this library
// runs on are alike); asked once, since the question takes longer than a launch.
template <class K>
int per_sm(K kernel, int threads) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  return std::max(1, n);
}

template <bool kRms>
gemm_status_t norm(gemm_ops_s* h, const void* x, int64_t ldx, const void* weight, const void* bias, void* y, int64_t ldy,
                   float* stats, int64_t T, int64_t D, float eps, gemm_dtype_t dtype, gemm_dtype_t wtype, void* stream) {
  gemm_status_t st = check_norm(h, T, D, dtype, wtype);
  if (st != GEMM_OK) return st;
  if (!(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  if (T == 0) return GEMM_OK;
  const int64_t e = bytes_of(dtype), ew = bytes_of(wtype), ns = kRms ? 4 : 8;
  if ((st = check_rows(x, ldx, D, e)) != GEMM_OK || (st = check_rows(y, ldy, D, e)) != GEMM_OK) return st;
  for (auto [p, a] : {std::pair<const void*, int64_t>(weight, ew), {bias, ew}, {stats, 4}})
    if (reinterpret_cast<uintptr_t>(p) % a) return GEMM_ERR_ALIGNMENT;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const Buf bufs[] = {{x, T, D * e, ldx * e, false},
                      {weight, weight ? 1 : 0, D * ew, D * ew, false},
                      {bias, bias ? 1 : 0, D * ew, D * ew, false},
                      {y, T, D * e, ldy * e, true},
                      {stats, stats ? T : 0, ns, ns, true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  NormArgs a = {};
  a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.stats = stats;
  a.ldx = ldx, a.ldy = ldy, a.T = T, a.D = D, a.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = vectors(16, D, e, {{x, ldx}, {y, ldy}}) && aligned16(weight) && aligned16(bias);
  const bool words = vectors(4, D, e, {{x, ldx}, {y, ldy}});
  return with_types(dtype, wtype, [&](auto tx, auto tw) {
    typedef decltype(tx) X;
    typedef decltype(tw) W;
    gemm_status_t st = GEMM_OK;
    auto rows = [&](auto vec, auto team, auto per, auto teams) {
      auto kernel = norm_rows<X, W, kRms, vec, team, per, teams>;
      static const int fit = per_sm(kernel, team * teams);
      const int64_t blocks = std::min<int64_t>(cdiv(T, teams), fit * h->num_sms);
      st = launch(h, kernel, dim3(static_cast<unsigned>(blocks)), dim3(team * teams), 0, 1, s, a);
      return true;
    };
    constexpr int kVec = 16 / sizeof(X);
    if (vec && with_team<4>(D / kVec, [&](auto... v) { return rows(Int<kVec>(), v...); })) return st;
    if constexpr (kVec == 8)
      if (!vec && words && with_team<8>(D / 2, [&](auto... v) { return rows(Int<2>(), v...); })) return st;
    if (!vec && with_team<8>(D, [&](auto... v) { return rows(Int<1>(), v...); })) return st;
    return launch(h, norm_any<X, W, kRms>, dim3(static_cast<unsigned>(T)), dim3(row_threads(D)), 0, 1, s, a);
  });
}

}  // namespace

extern "C" {

gemm_status_t gemm_layer_norm(gemm_ops_t h, const void* x, int64_t ldx, const void* weight, const void* bias, void* y,
                              int64_t ldy, float* stats, int64_t T, int64_t D, float eps, gemm_dtype_t dtype,
                              gemm_dtype_t wtype, void* stream) {
  return norm<false>(h, x, ldx, weight, bias, y, ldy, stats, T, D, eps, dtype, wtype, stream);
}

gemm_status_t gemm_rms_norm(gemm_ops_t h, const void* x, int64_t ldx, const void* weight, void* y, int64_t ldy,
                            float* stats, int64_t T, int64_t D, float eps, gemm_dtype_t dtype, gemm_dtype_t wtype,
                            void* stream) {
  return norm<true>(h, x, ldx, weight, nullptr, y, ldy, stats, T, D, eps, dtype, wtype, stream);
}

}  // extern "C"
