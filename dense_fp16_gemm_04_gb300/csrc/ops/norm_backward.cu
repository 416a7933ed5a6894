// norm_backward.cu -- host side of the norms' gradients.
#include "norm_host.cuh"

namespace {

using namespace gb300::ops;

constexpr int kBackSmem = 200 * 1024;  // the largest ring of norm_rows_back: 192 KB

// Allows a kernel kBackSmem bytes of shared memory, once on each device (`done`: a bit
// for each of the first 64).
template <class K>
bool allow_smem(const gemm_ops_s* h, K kernel, std::atomic<uint64_t>& done) {
  const uint64_t bit = h->device < 64 ? 1ull << h->device : 0;
  if (done.load() & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBackSmem) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done |= bit;
  return true;
}

// Chunks of rows whose sums are taken apart by norm_dw_any: enough blocks of 32
// columns for the device, of at least 32 rows.
int64_t row_chunks(const gemm_ops_s* h, int64_t T, int64_t D) {
  return std::max<int64_t>(1, std::min(cdiv(T, 32), cdiv(8 * h->num_sms, cdiv(D, 32))));
}

// Blocks of norm_rows_back, of `teams` teams: one to an SM, or kBackThreads threads of
// them, each with at least two rows a team for its one row of sums.
constexpr int kBackThreads = 512;
int64_t back_blocks(const gemm_ops_s* h, int64_t T, int team, int teams) {
  return std::max<int64_t>(1, std::min<int64_t>(cdiv(T, 2 * teams), h->num_sms * std::max(1, kBackThreads / (team * teams))));
}
// The most of either.
int64_t most_chunks(const gemm_ops_s* h, int64_t T, int64_t D) {
  return std::max(row_chunks(h, T, D), std::min<int64_t>(cdiv(T, 2), 2 * h->num_sms));
}

template <bool kRms>
gemm_status_t norm_backward(gemm_ops_s* h, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                            const float* stats, void* dx, int64_t lddx, void* dweight, void* dbias, void* workspace,
                            size_t workspace_bytes, int64_t T, int64_t D, gemm_dtype_t dtype, gemm_dtype_t wtype,
                            void* stream) {
  gemm_status_t st = check_norm(h, T, D, dtype, wtype);
  if (st != GEMM_OK) return st;
  const int64_t e = bytes_of(dtype), ew = bytes_of(wtype), ns = kRms ? 4 : 8;
  for (auto [p, ld] : {std::pair<const void*, int64_t>(dy, lddy), {x, ldx}, {dx, lddx}})
    if ((st = check_rows(p, ld, D, e)) != GEMM_OK) return st;
  for (auto [p, a] : {std::pair<const void*, int64_t>(weight, ew), {dweight, ew}, {dbias, ew}, {stats, 4}, {workspace, 256}})
    if (reinterpret_cast<uintptr_t>(p) % a) return GEMM_ERR_ALIGNMENT;
  const size_t need = gemm_norm_backward_workspace(h, T, D);
  if (workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const Buf bufs[] = {{dy, T, D * e, lddy * e, false},
                      {x, T, D * e, ldx * e, false},
                      {weight, weight ? 1 : 0, D * ew, D * ew, false},
                      {stats, T, ns, ns, false},
                      {dx, T, D * e, lddx * e, true},
                      {dweight, dweight ? 1 : 0, D * ew, D * ew, true},
                      {dbias, dbias ? 1 : 0, D * ew, D * ew, true},
                      {workspace, need ? 1 : 0, static_cast<int64_t>(need), static_cast<int64_t>(need), true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no row, no gradient
    for (void* p : {dweight, dbias})
      if (p && cudaMemsetAsync(p, 0, D * ew, s) != cudaSuccess) return GEMM_ERR_CUDA;
    return GEMM_OK;
  }
  NormArgs a = {};
  a.x = x, a.dy = dy, a.weight = weight, a.y = dx, a.stats = const_cast<float*>(stats);
  a.ldx = ldx, a.lddy = lddy, a.ldy = lddx, a.T = T, a.D = D;
  a.partial = static_cast<float*>(workspace);
  a.chunks = row_chunks(h, T, D);
  a.dweight = dweight, a.dbias = dbias;
  const bool vec = vectors(16, D, e, {{x, ldx}, {dy, lddy}, {dx, lddx}}) && aligned16(weight);
  const bool words = vectors(4, D, e, {{x, ldx}, {dy, lddy}, {dx, lddx}});
  return with_types(dtype, wtype, [&](auto tx, auto tw) {
    typedef decltype(tx) X;
    typedef decltype(tw) W;
    const bool sums = dweight || dbias;
    gemm_status_t st = GEMM_OK;
    if (!sums) a.partial = nullptr;
    auto rows = [&](auto vec, auto team, auto per, auto teams) {
      a.chunks = back_blocks(h, T, team, teams);
      const size_t sums_bytes = teams > 1 ? 2 * D * sizeof(float) : 0;
      const dim3 grid(static_cast<unsigned>(a.chunks)), block(team * teams);
      // (1024 threads have no registers for the next row of pairs.)
      if constexpr (vec == 1 || (vec == 2 && team < 1024)) {
        st = launch(h, norm_rows_back_single<X, W, kRms, vec, team, per, teams>, grid, block, sums_bytes, 1, s, a);
      } else {
        auto kernel = norm_rows_back<X, W, kRms, vec, team, per, teams>;
        static std::atomic<uint64_t> allowed{0};
        st = allow_smem(h, kernel, allowed)
                 ? launch(h, kernel, grid, block, std::max(back_ring<X, vec, per>(team * teams), sums_bytes), 1, s, a)
                 : GEMM_ERR_CUDA;
      }
      return true;
    };
    constexpr int kVec = 16 / sizeof(X), kWord = 4 / sizeof(X);
    // 16 bytes at a time, 4, or an element: 1530 x 7642 bf16 (words) 21 us, 36 by elements.
    auto with_back = [&](auto f) {  // a team for whole vectors
      const int64_t n = D / kVec;
      // One sum a column, or fp32 rows, leave registers for four vectors a thread, and so
      // for two teams of 8192 columns on an SM, which wait for their sums apart: RMS norm of
      // 8192 x 8192 bf16 75 -> 67 us, layer norm of 4096 x 8192 fp32 73 -> 66.
      if constexpr (kRms || kVec == 4) {
        if (n <= 32) return f(Int<32>(), Int<1>(), Int<8>());
        if (n <= 64) return f(Int<32>(), Int<2>(), Int<8>());
        if (n <= 128) return f(Int<32>(), Int<4>(), Int<8>());
        if (n <= 256) return f(Int<64>(), Int<4>(), Int<4>());
        if (n <= 512) return f(Int<128>(), Int<4>(), Int<2>());
        if (n <= 1024) return f(Int<256>(), Int<4>(), Int<1>());
        if (n <= 2048) return f(Int<512>(), Int<4>(), Int<1>());
        return false;
      } else {
        return with_team<2>(n, f);
      }
    };
    if (!(vec && with_back([&](auto... v) { return rows(Int<kVec>(), v...); })) &&
        !(!vec && words && with_team<8>(D / kWord, [&](auto... v) { return rows(Int<kWord>(), v...); })) &&
        !(!vec && !words && with_team<8>(D, [&](auto... v) { return rows(Int<1>(), v...); }))) {
      st = launch(h, norm_dx_any<X, W, kRms>, dim3(static_cast<unsigned>(T)), dim3(row_threads(D)), 0, 1, s, a);
      if (st == GEMM_OK && sums)
        st = launch(h, norm_dw_any<X, kRms>, dim3(static_cast<unsigned>(cdiv(D, 32)), static_cast<unsigned>(a.chunks)),
                    dim3(256), 0, 1, s, a);
    }
    if (st != GEMM_OK || !sums) return st;
    // More groups where there are few blocks: RMS norm of 16384 x 2048 37.8 -> 36.8 us, but
    // layer norm of 8192 x 8192 77.1 -> 79.8.
    const dim3 grid(static_cast<unsigned>(cdiv(D, 32)), dbias ? 2 : 1);
    return static_cast<int64_t>(grid.x) * grid.y <= h->num_sms ? launch(h, norm_dw_sum<W, 32>, grid, dim3(32 * 32), 0, 1, s, a)
                                         : launch(h, norm_dw_sum<W, 16>, grid, dim3(32 * 16), 0, 1, s, a);
  });
}

}  // namespace

extern "C" {

size_t gemm_norm_backward_workspace(gemm_ops_t h, int64_t T, int64_t D) {
  if (!h || T <= 0 || D <= 0 || !dim_ok(T) || !dim_ok(D)) return 0;
  return most_chunks(h, T, D) * 2 * D * sizeof(float);
}

gemm_status_t gemm_layer_norm_backward(gemm_ops_t h, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                       const void* weight, const float* stats, void* dx, int64_t lddx, void* dweight,
                                       void* dbias, void* workspace, size_t workspace_bytes, int64_t T, int64_t D,
                                       gemm_dtype_t dtype, gemm_dtype_t wtype, void* stream) {
  return norm_backward<false>(h, dy, lddy, x, ldx, weight, stats, dx, lddx, dweight, dbias, workspace, workspace_bytes, T,
                              D, dtype, wtype, stream);
}

gemm_status_t gemm_rms_norm_backward(gemm_ops_t h, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                     const void* weight, const float* stats, void* dx, int64_t lddx, void* dweight,
                                     void* workspace, size_t workspace_bytes, int64_t T, int64_t D, gemm_dtype_t dtype,
                                     gemm_dtype_t wtype, void* stream) {
  return norm_backward<true>(h, dy, lddy, x, ldx, weight, stats, dx, lddx, dweight, nullptr, workspace, workspace_bytes,
                             T, D, dtype, wtype, stream);
}

}  // extern "C"
