// norm_host.cuh -- what the host sides of the norms' two passes share: types, checks
// and the choice of a team for a row's length.
#pragma once
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "host.cuh"
#include "norm_kernels.cuh"

namespace gb300 {
namespace ops {

// f(x's type, the weight's): the weight is of x's type or fp32.
template <class F>
gemm_status_t with_types(gemm_dtype_t dtype, gemm_dtype_t wtype, F f) {
  switch (dtype) {
    case GEMM_F16: return wtype == GEMM_F32 ? f(__half(), float()) : f(__half(), __half());
    case GEMM_BF16: return wtype == GEMM_F32 ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
    default: return f(float(), float());
  }
}

inline int64_t bytes_of(gemm_dtype_t t) { return t == GEMM_F32 ? 4 : 2; }

inline gemm_status_t check_norm(const gemm_ops_s* h, int64_t T, int64_t D, gemm_dtype_t dtype, gemm_dtype_t wtype) {
  if (!h || !dim_ok(T) || !dim_ok(D) || D == 0) return GEMM_ERR_INVALID_ARG;
  if (dtype != GEMM_F16 && dtype != GEMM_BF16 && dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
  return wtype == dtype || wtype == GEMM_F32 ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

// Rows of D elements ld apart at an element's alignment.
inline gemm_status_t check_rows(const void* p, int64_t ld, int64_t D, int64_t e) {
  if (ld < D || ld >= (1ll << 30)) return GEMM_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % e ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

// Whether rows of D elements of e bytes may be read `bytes` at a time.
inline bool vectors(int64_t bytes, int64_t D, int64_t e, std::initializer_list<std::pair<const void*, int64_t>> rows) {
  bool ok = D * e % bytes == 0;
  for (auto [p, ld] : rows) ok = ok && reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * e % bytes == 0;
  return ok;
}

template <int kV>
using Int = std::integral_constant<int, kV>;

// f(team, vectors a thread, teams) for rows of n vectors: the smallest team that
// holds one, false for none.
template <int kMostPer, class F>
bool with_team(int64_t n, F f) {
  if (n <= 32) return f(Int<32>(), Int<1>(), Int<8>());
  if (n <= 64) return f(Int<32>(), Int<2>(), Int<8>());
  if constexpr (kMostPer > 2)
    if (n <= 32 * kMostPer) return f(Int<32>(), Int<kMostPer>(), Int<8>());
  if constexpr (kMostPer < 8)
    if (n <= 256) return f(Int<128>(), Int<2>(), Int<2>());
  if constexpr (kMostPer > 2)
    if (n <= 128 * kMostPer) return f(Int<128>(), Int<kMostPer>(), Int<2>());
  if (n <= 256 * kMostPer) return f(Int<256>(), Int<kMostPer>(), Int<1>());
  if (n <= 512 * kMostPer) return f(Int<512>(), Int<kMostPer>(), Int<1>());
  if (n <= 1024 * kMostPer) return f(Int<1024>(), Int<kMostPer>(), Int<1>());
  return false;
}

inline unsigned row_threads(int64_t D) { return static_cast<unsigned>(std::min<int64_t>(512, up(D, 32))); }

}  // namespace ops
}  // namespace gb300
