// ops.cu -- host side of the C ABI declared in include/gemm_ops.h: argument
// checks, tensor maps, the choice of kernel and the launches.
#include "host.cuh"
#include "ortho_kernels.cuh"
#include "stream_kernel.cuh"

namespace {

using namespace gb300::ops;

// Tokens of the streaming products of 16-bit weights; more go to the tensor
// cores' own products.  16 and 17 tokens: weights of 1024 x 4096 11.4 and 13.7
// us, 2048 x 5632 22.1 and 25.3 us, 4096 x 8192 46.3 and 41.7 us, 8192 x 16384
// 145 and 133 us.
constexpr int64_t kMaxStreamTokens = 16;

// out = A B^T, rounded to 16 bits.
gemm_status_t product(gemm_ops_s* h, const Product& p, const Stack& out, int early, cudaStream_t stream) {
  FusedArgs a = base_args(h, p);
  a.early = early;
  return fused<kEpiStore>(h, p, a, out, {}, stream);
}

// How a product of few tokens is laid out: warps per CTA, CTAs per k-slice,
// k-slices, and the CTA's shared memory.
struct StreamPlan {
  int64_t warps, ctas, slices, ring;
  size_t smem;
};

constexpr size_t kStreamSmem = 226 * 1024;
constexpr int64_t kMaxSlices = 65535;  // a grid's second dimension

// 8-column tiles per CTA.
template <int kW>
int stream_tiles(int64_t T) {
  return T <= stream_tokens(kW) ? 1 : 2;
}

template <int kW, bool kGlu>
StreamPlan stream_plan(const gemm_ops_s* h, int64_t T, int64_t N, int64_t K) {
  StreamPlan p;
  const int64_t bk = stream_block_k(kW), blocks = cdiv(K, bk), tiles = cdiv(N, stream_tile(kGlu));
  const int64_t nt = stream_tiles<kW>(T), held = std::min(T, nt * stream_tokens(kW));
  // Enough warps that each keeps a block or two of a tile; the rest of the
  // parallelism comes from tiles, or from cutting K where they are few.
  p.warps = blocks >= 16 ? 16 : blocks >= 8 ? 8 : 4;
  auto smem = [&] {  // the warps' sums, their blocks in flight, and x
    return static_cast<size_t>(p.warps) * (2 * 2 * nt * 128 * sizeof(float) + p.ring * stream_slot_bytes(kW)) +
           static_cast<size_t>(cdiv(blocks, p.slices)) * bk * held * 2 + kStreamHead;
  };
  for (;; p.warps /= 2) {
    p.ring = kStreamMaxRing;
    p.slices = std::max<int64_t>(1, std::min(h->num_sms / tiles, blocks / (2 * p.warps)));
    while (p.ring > 2 && smem() > kStreamSmem) --p.ring;
    while (p.slices < blocks && smem() > kStreamSmem) ++p.slices;
    // The longest rows of many tokens: fewer warps leave room for more of x in
    // each slice (2^28 codes a row, 16 tokens: 104858 slices with 16, 55189 with 8).
    if (p.slices <= kMaxSlices || p.warps == 4) break;
  }
  while (p.ring < kStreamMaxRing) {  // what the slices freed
    ++p.ring;
    if (smem() > kStreamSmem) {
      --p.ring;
      break;
    }
  }
  p.smem = smem();
  const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(16 / p.warps, kStreamSmem / p.smem));
  p.ctas = std::min(tiles, std::max<int64_t>(1, per_sm * h->num_sms / p.slices));
  return p;
}

// The kernel's offsets into W are 32 bits: rows of one launch, 4 GB at most and
// a whole number of tiles (a row has at most kMaxStreamRow bytes).
constexpr int64_t kMaxStreamRow = 1 << 27;
int64_t stream_rows(int64_t row_bytes) { return (1ll << 32) / row_bytes / 32 * 32; }

template <int kW, bool kGlu>
size_t stream_partial_bytes(const gemm_ops_s* h, int64_t T, int64_t N, int64_t K) {
  if (kW != kW16) N = std::min(N, stream_rows(K / 2));
  const StreamPlan p = stream_plan<kW, kGlu>(h, T, N, K);
  return p.slices > 1 ? static_cast<size_t>(p.slices) * T * N * (kGlu ? 2 : 1) * 4 : 0;
}

// Whether a block's weights (rows ld 16-bit elements apart) suit one launch.
bool stream_fits(int64_t rows, int64_t ld) { return 2 * ld <= kMaxStreamRow && rows <= stream_rows(2 * ld); }

typedef void (*StreamKernel)(const StreamArgs);

template <int kW, bool kGlu>
StreamKernel stream_variant(bool bf16, int nt) {
  if constexpr (stream_groups(kW) > 1)
    return bf16 ? stream_kernel<true, kW, kGlu, 1> : stream_kernel<false, kW, kGlu, 1>;
  else if (nt == 1)
    return bf16 ? stream_kernel<true, kW, kGlu, 1> : stream_kernel<false, kW, kGlu, 1>;
  else
    return bf16 ? stream_kernel<true, kW, kGlu, 2> : stream_kernel<false, kW, kGlu, 2>;
}

// The products of a.cols columns; `a` is complete but for N and the up rows.
template <int kW, bool kGlu>
gemm_status_t stream_product(gemm_ops_s* h, StreamArgs a, bool bf16, cudaStream_t stream) {
  const int64_t row_bytes = a.ldw * (kW == kW16 ? 2 : 1), groups = kW == kW16 ? 0 : a.K >> a.group_shift;
  a.up_w = a.cols * row_bytes;
  a.up_s = a.cols * groups;
  const int64_t most = stream_rows(row_bytes), cols = a.cols;
  const int nt = stream_tiles<kW>(a.T);
  const StreamPlan p = stream_plan<kW, kGlu>(h, a.T, std::min(cols, most), a.K);
  a.ring = static_cast<int32_t>(p.ring);
  for (int64_t n0 = 0; n0 < cols; n0 += most) {
    a.N = static_cast<int32_t>(std::min(most, cols - n0));
    const int64_t ctas = std::min<int64_t>(p.ctas, cdiv(a.N, stream_tile(kGlu)));
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(p.slices),
                    static_cast<unsigned>(cdiv(a.T, nt * stream_tokens(kW))));
    const dim3 block(static_cast<unsigned>(32 * p.warps));
    gemm_status_t st = launch(h, stream_variant<kW, kGlu>(bf16, nt), grid, block, p.smem, 1, stream, a);
    if (st == GEMM_OK && p.slices > 1) {
      const int64_t n = std::min<int64_t>(cdiv(static_cast<int64_t>(a.T) * a.N, 256), 8 * h->num_sms);
      st = launch(h, stream_reduce<kGlu>, dim3(static_cast<unsigned>(n)), dim3(256), 0, 1, stream, a,
                  static_cast<int32_t>(p.slices), static_cast<int32_t>(bf16));
    }
    if (st != GEMM_OK) return st;
    a.w = static_cast<const char*>(a.w) + most * row_bytes;
    a.y += most;
    if (a.gu) a.gu += most;
    if (a.scales) a.scales += most * groups;
    if (a.zeros) a.zeros += most * groups;
  }
  return GEMM_OK;
}

template <int kW, bool kGlu>
bool set_stream_attr() {
  for (bool bf16 : {false, true})
    for (int nt : {1, 2})
      if (cudaFuncSetAttribute(stream_variant<kW, kGlu>(bf16, nt), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kStreamSmem) != cudaSuccess)
        return false;
  return true;
}

// The forms of small groups for few tokens: as many as one 8-column tile holds.
// 8192 x 8192 codes, 3 tokens in groups of 32: by columns (two tiles) 22.9 us, in
// turn 22.3 us; 4 and 5 in groups of 64: by columns 17.9 (one tile) and 22.3 us,
// in turn 18.1 and 18.4 us.
constexpr int64_t kFewG32 = stream_tokens(kW4G32Few), kFewG64 = stream_tokens(kW4G64Few);

constexpr int64_t kMaxW4Tokens = 8 * 65535;  // tiles of 8 and more in a grid's third dimension

template <bool kGlu>
size_t w4_workspace(gemm_ops_s* h, int64_t T, int64_t N, int64_t K) {
  // No group divides any other K: the product refuses it.
  if (!h || T <= 0 || N <= 0 || K <= 0 || K % 32 != 0 || K / 2 > kMaxStreamRow || T > kMaxW4Tokens)
    return 0;
  // Whatever the groups.
  return std::max({T <= kFewG32 ? stream_partial_bytes<kW4G32Few, kGlu>(h, T, N, K)
                                : stream_partial_bytes<kW4G32, kGlu>(h, T, N, K),
                   T <= kFewG64 ? stream_partial_bytes<kW4G64Few, kGlu>(h, T, N, K)
                                : stream_partial_bytes<kW4G64, kGlu>(h, T, N, K),
                   stream_partial_bytes<kW4G128, kGlu>(h, T, N, K)});
}

template <bool kGlu>
gemm_status_t w4_product(gemm_ops_s* h, const StreamArgs& a, int64_t group, bool bf16, cudaStream_t s) {
  if (group == 32)
    return a.T <= kFewG32 ? stream_product<kW4G32Few, kGlu>(h, a, bf16, s) : stream_product<kW4G32, kGlu>(h, a, bf16, s);
  if (group == 64)
    return a.T <= kFewG64 ? stream_product<kW4G64Few, kGlu>(h, a, bf16, s) : stream_product<kW4G64, kGlu>(h, a, bf16, s);
  return stream_product<kW4G128, kGlu>(h, a, bf16, s);
}

template <int kSplit>
bool set_split_attr() {
  if constexpr (kSplit < 8) {
    if (!set_attr<Lone<kEpiSplit, kSplit>>() || !set_attr<Lone<kEpiSplitSym, kSplit>>() ||
        !set_attr<Lone<kEpiSplit, 1, kSplit>>() || !set_attr<Lone<kEpiSplitSym, 1, kSplit>>())
      return false;
  }
  return set_attr<Lone<kEpiStore, kSplit>>() && set_attr<Lone<kEpiGlu, kSplit>>() &&
         set_attr<Lone<kEpiGluBwd, kSplit>>();
}

bool ffn_dims_ok(int64_t T, int64_t D, int64_t F) {
  return dim_ok(T) && dim_ok(D) && dim_ok(F) && F <= INT32_MAX / 2;
}

// Checks shared by the block's two passes.
gemm_status_t check_ffn(const gemm_ops_s* h, int64_t T, int64_t D, int64_t F, gemm_act_t act,
                        gemm_dtype_t dtype) {
  if (!h || !ffn_dims_ok(T, D, F)) return GEMM_ERR_INVALID_ARG;
  if (act < GEMM_ACT_SILU || act > GEMM_ACT_RELU) return GEMM_ERR_INVALID_ARG;
  if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
  if (D % 8 != 0 || F % 8 != 0) return GEMM_ERR_ALIGNMENT;
  return GEMM_OK;
}

// Rows of the hidden tensors in workspaces, elements apart: whole 128-byte
// lines, so that no load of them straddles two.
int64_t hidden_pitch(int64_t F) { return up(F, 64); }
// Bytes of h; the backward pass's workspace is dg and du (rows of two pitches),
// then h.
size_t hidden_bytes(int64_t T, int64_t F) { return up(T * hidden_pitch(F) * 2, 256); }

struct OrthoSpace {
  int64_t r, pitch, pitch_r;  // r: order of the Gram matrix
  size_t x0, x1, p, q, partial, total;
};
OrthoSpace ortho_space(int64_t batch, int64_t M, int64_t N) {
  OrthoSpace s;
  s.r = std::min(M, N);
  s.pitch = up(N, 8);
  s.pitch_r = up(s.r, 8);
  const size_t xb = up(batch * 2 * M * s.pitch * 2, 256), pb = up(batch * 2 * s.r * s.pitch_r * 2, 256);
  s.x0 = 0;
  s.x1 = xb;
  s.p = 2 * xb;
  s.q = s.p + pb;
  s.partial = s.q + pb;
  s.total = s.partial + up(batch * kNormBlocks * 4, 256);
  return s;
}

}  // namespace

extern "C" {

gemm_status_t gemm_ops_create(gemm_ops_t* out, int device) {
  if (!out) return GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) return GEMM_ERR_CUDA;
  if (device < 0 || device >= ndev) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(device);
  if (!g.ok) return GEMM_ERR_CUDA;
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return GEMM_ERR_CUDA;
  if (major != 10 || minor != 3) return GEMM_ERR_UNSUPPORTED_DEVICE;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !fn)
    return GEMM_ERR_CUDA;
  if (!set_attr<Pair<kEpiStore>>() || !set_attr<Pair<kEpiGlu>>() || !set_attr<Pair<kEpiGluBwd>>() ||
      !set_attr<Pair<kEpiSplit>>() || !set_attr<Pair<kEpiSplitSym>>() || !set_attr<Lone<kEpiStore>>() ||
      !set_attr<Lone<kEpiGlu>>() || !set_attr<Lone<kEpiGluBwd>>() || !set_attr<Lone<kEpiSplit>>() ||
      !set_attr<Lone<kEpiSplitSym>>() ||
      !set_attr<TwoPairs<kEpiStore>>() || !set_attr<TwoPairs<kEpiGlu>>() || !set_attr<TwoPairs<kEpiGluBwd>>() ||
      !set_attr<TwoPairs<kEpiSplit>>() || !set_attr<TwoPairs<kEpiSplitSym>>() || !set_split_attr<2>() ||
      !set_split_attr<4>() || !set_split_attr<8>() ||
      !set_stream_attr<kW16, false>() || !set_stream_attr<kW16, true>() ||
      !set_stream_attr<kW4G32, false>() || !set_stream_attr<kW4G32, true>() ||
      !set_stream_attr<kW4G64, false>() || !set_stream_attr<kW4G64, true>() ||
      !set_stream_attr<kW4G128, false>() || !set_stream_attr<kW4G128, true>() ||
      !set_stream_attr<kW4G32Few, false>() || !set_stream_attr<kW4G32Few, true>() ||
      !set_stream_attr<kW4G64Few, false>() || !set_stream_attr<kW4G64Few, true>())
    return GEMM_ERR_CUDA;
  gemm_ops_s* h = new (std::nothrow) gemm_ops_s();
  if (!h) return GEMM_ERR_OOM;
  h->device = device;
  h->num_sms = sms;
  h->encode = fn;
  h->max_pairs = std::min({max_clusters<Pair<kEpiStore>>(), max_clusters<Pair<kEpiGlu>>(),
                           max_clusters<Pair<kEpiGluBwd>>(), max_clusters<Pair<kEpiSplit>>(),
                           max_clusters<Pair<kEpiSplitSym>>()});
  h->max_twos = std::min({max_clusters<TwoPairs<kEpiStore>>(), max_clusters<TwoPairs<kEpiGlu>>(),
                          max_clusters<TwoPairs<kEpiGluBwd>>(), max_clusters<TwoPairs<kEpiSplit>>(),
                          max_clusters<TwoPairs<kEpiSplitSym>>()});
  h->max_split[1] = max_clusters<Lone<kEpiStore, 2>>();
  h->max_split[2] = max_clusters<Lone<kEpiStore, 4>>();
  h->max_split[3] = max_clusters<Lone<kEpiStore, 8>>();
  if (!xent_setup(h)) {
    delete h;
    return GEMM_ERR_CUDA;
  }
  if (cudaMalloc(&h->d_err, sizeof(h->last_err)) != cudaSuccess) {
    delete h;
    return GEMM_ERR_OOM;
  }
  if (cudaMemset(h->d_err, 0, sizeof(h->last_err)) != cudaSuccess) {
    cudaFree(h->d_err);
    delete h;
    return GEMM_ERR_CUDA;
  }
  *out = h;
  return GEMM_OK;
}

gemm_status_t gemm_ops_destroy(gemm_ops_t h) {
  if (!h) return GEMM_OK;
  DeviceGuard g(h->device);
  if (h->d_err) cudaFree(h->d_err);
  delete h;
  return GEMM_OK;
}

gemm_status_t gemm_ops_check_error(gemm_ops_t h) {
  if (!h) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  uint32_t rec[4] = {0, 0, 0, 0};
  if (cudaDeviceSynchronize() != cudaSuccess) return GEMM_ERR_CUDA;
  if (cudaMemcpy(rec, h->d_err, sizeof(rec), cudaMemcpyDeviceToHost) != cudaSuccess)
    return GEMM_ERR_CUDA;
  if (rec[0] == 0) return GEMM_OK;
  std::memcpy(h->last_err, rec, sizeof(rec));
  if (cudaMemset(h->d_err, 0, sizeof(rec)) != cudaSuccess) return GEMM_ERR_CUDA;
  return static_cast<gemm_status_t>(rec[0]);
}

gemm_status_t gemm_ops_last_error_detail(gemm_ops_t h, uint32_t detail[4]) {
  if (!h || !detail) return GEMM_ERR_INVALID_ARG;
  std::memcpy(detail, h->last_err, sizeof(h->last_err));
  return GEMM_OK;
}

gemm_status_t gemm_ops_set_watchdog(gemm_ops_t h, uint64_t timeout_ns, int32_t skip_k_block) {
  if (!h || skip_k_block < -1) return GEMM_ERR_INVALID_ARG;
  h->timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;
  h->skip_kb = skip_k_block;
  return GEMM_OK;
}

uint64_t gemm_ops_launch_count(gemm_ops_t h) { return h ? h->launches.load() : 0; }

size_t gemm_gated_ffn_workspace(gemm_ops_t h, int64_t T, int64_t D, int64_t F) {
  if (!h || T <= 0 || D <= 0 || F <= 0 || !ffn_dims_ok(T, D, F)) return 0;
  size_t s = hidden_bytes(T, F);
  if (T <= kMaxStreamTokens)
    s += std::max(stream_partial_bytes<kW16, true>(h, T, F, D), stream_partial_bytes<kW16, false>(h, T, D, F));
  return s;
}

gemm_status_t gemm_gated_ffn(gemm_ops_t h, const void* x, int64_t ldx, const void* w_in,
                             int64_t ldw_in, const void* w_down, int64_t ldw_down, void* y,
                             int64_t ldy, void* gu, void* workspace, size_t workspace_bytes, int64_t T,
                             int64_t D, int64_t F, gemm_act_t act, gemm_dtype_t dtype, void* stream) {
  gemm_status_t st = check_ffn(h, T, D, F, act, dtype);
  if (st != GEMM_OK) return st;
  if (T == 0) return GEMM_OK;
  if (D == 0) {  // y has no elements; g and u are empty sums
    if (!gu || F == 0) return GEMM_OK;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    if (!on_device(gu, h->device)) return GEMM_ERR_INVALID_ARG;
    return cudaMemsetAsync(gu, 0, T * 4 * F, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK
                                                                                              : GEMM_ERR_CUDA;
  }
  for (auto [ld, cols] : {std::pair<int64_t, int64_t>(ldx, D), {ldw_in, D}, {ldw_down, F}, {ldy, D}})
    if ((st = check_ld(ld, cols)) != GEMM_OK) return st;
  if (!aligned16(x) || !aligned16(w_in) || !aligned16(w_down) || !aligned16(y) || !aligned16(gu) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GEMM_ERR_ALIGNMENT;
  const size_t need = gemm_gated_ffn_workspace(h, T, D, F);
  if (workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const Buf bufs[] = {{x, T, D * 2, ldx * 2, false},
                      {w_in, 2 * F, D * 2, ldw_in * 2, false},
                      {w_down, F > 0 ? D : 0, F * 2, ldw_down * 2, false},
                      {y, T, D * 2, ldy * 2, true},
                      {gu, gu ? T : 0, 4 * F, 4 * F, true},
                      {workspace, 1, static_cast<int64_t>(need), static_cast<int64_t>(need), true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (F == 0)
    return cudaMemset2DAsync(y, ldy * 2, 0, D * 2, T, s) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  const bool bf16 = dtype == GEMM_BF16;
  void* hid = workspace;
  const int64_t pf = hidden_pitch(F);
  void* partial = static_cast<char*>(workspace) + hidden_bytes(T, F);
  if (T <= kMaxStreamTokens && stream_fits(F, ldw_in) && stream_fits(D, ldw_down)) {
    StreamArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.w = w_in;
    a.ldw = ldw_in;
    a.y = static_cast<uint16_t*>(hid);
    a.ldy = pf;
    a.gu = static_cast<uint16_t*>(gu);
    a.partial = static_cast<float*>(partial);
    a.T = static_cast<int32_t>(T);
    a.K = static_cast<int32_t>(D);
    a.cols = static_cast<int32_t>(F);
    a.act = act;
    if ((st = stream_product<kW16, true>(h, a, bf16, s)) != GEMM_OK) return st;
    a.x = static_cast<const uint16_t*>(hid);
    a.ldx = pf;
    a.w = w_down;
    a.ldw = ldw_down;
    a.y = static_cast<uint16_t*>(y);
    a.ldy = ldy;
    a.gu = nullptr;
    a.early = 1;  // the kernels above wrote neither W nor what they waited for
    a.K = static_cast<int32_t>(F);
    a.cols = static_cast<int32_t>(D);
    return stream_product<kW16, false>(h, a, bf16, s);
  }
  const Product p = {T, F, D, {x, T, D, ldx, 1, T * ldx}, {w_in, F, D, ldw_in, 2, F * ldw_in},
                     false, false, bf16, 1, 1};
  FusedArgs a = base_args(h, p);
  a.act = act;
  a.save = gu != nullptr;
  const Stack keep = {gu, T, F, 2 * F, 2, F}, hs = {hid, T, F, pf, 1, T * pf};
  st = fused<kEpiGlu>(h, p, a, hs, gu ? keep : Stack{}, s);
  if (st != GEMM_OK) return st;
  const Product down = {T, D, F, hs, {w_down, D, F, ldw_down, 1, D * ldw_down}, false, false, bf16, 1, 1};
  return product(h, down, {y, T, D, ldy, 1, T * ldy}, kEarlyB, s);
}

size_t gemm_gated_ffn_backward_workspace(gemm_ops_t h, int64_t T, int64_t D, int64_t F) {
  if (!h || T <= 0 || D <= 0 || F <= 0 || !ffn_dims_ok(T, D, F)) return 0;
  return 3 * hidden_bytes(T, F);
}

gemm_status_t gemm_gated_ffn_backward(gemm_ops_t h, const void* dy, int64_t lddy, const void* x,
                                      int64_t ldx, const void* w_in, int64_t ldw_in,
                                      const void* w_down, int64_t ldw_down, const void* gu, void* dx,
                                      int64_t lddx, void* dw_in, void* dw_down, void* workspace,
                                      size_t workspace_bytes, int64_t T, int64_t D, int64_t F,
                                      gemm_act_t act, gemm_dtype_t dtype, void* stream) {
  gemm_status_t st = check_ffn(h, T, D, F, act, dtype);
  if (st != GEMM_OK) return st;
  if (D == 0) return GEMM_OK;
  for (auto [ld, cols] :
       {std::pair<int64_t, int64_t>(lddy, D), {ldx, D}, {ldw_in, D}, {ldw_down, F}, {lddx, D}})
    if ((st = check_ld(ld, cols)) != GEMM_OK) return st;
  for (const void* p : {dy, x, w_in, w_down, gu, static_cast<const void*>(dx), static_cast<const void*>(dw_in),
                        static_cast<const void*>(dw_down)})
    if (!aligned16(p)) return GEMM_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return GEMM_ERR_ALIGNMENT;
  const size_t need = gemm_gated_ffn_backward_workspace(h, T, D, F);
  if (workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const int64_t wrows = F > 0 ? D : 0;
  const Buf bufs[] = {{dy, T, D * 2, lddy * 2, false},
                      {x, T, D * 2, ldx * 2, false},
                      {w_in, 2 * F, D * 2, ldw_in * 2, false},
                      {w_down, wrows, F * 2, ldw_down * 2, false},
                      {gu, F > 0 ? T : 0, 4 * F, 4 * F, false},
                      {dx, T, D * 2, lddx * 2, true},
                      {dw_in, 2 * F, D * 2, D * 2, true},
                      {dw_down, wrows, F * 2, F * 2, true},
                      {workspace, need ? 1 : 0, static_cast<int64_t>(need), static_cast<int64_t>(need), true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (F == 0)
    return T == 0 || cudaMemset2DAsync(dx, lddx * 2, 0, D * 2, T, s) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  if (T == 0)  // no token, no gradient
    return cudaMemsetAsync(dw_in, 0, 4 * F * D, s) == cudaSuccess &&
                   cudaMemsetAsync(dw_down, 0, 2 * F * D, s) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
  const bool bf16 = dtype == GEMM_BF16;
  const int64_t pf = hidden_pitch(F);
  uint16_t* dgu = static_cast<uint16_t*>(workspace);
  uint16_t* hid = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + 2 * hidden_bytes(T, F));
  const Stack dys = {dy, T, D, lddy, 1, T * lddy};
  // dg and du are two matrices side by side, as are the halves of w_in one
  // after the other.
  const Stack hs = {hid, T, F, pf, 1, T * pf}, dgus = {dgu, T, F, 2 * pf, 2, pf};
  const Stack w_ins = {w_in, F, D, ldw_in, 2, F * ldw_in};
  // dh = dy Wd (Wd is stored [K, N] here), then dg, du and h.
  const Product ph = {T, F, D, dys, {w_down, D, F, ldw_down, 1, D * ldw_down}, false, true, bf16, 1, 1};
  FusedArgs a = base_args(h, ph);
  a.act = act;
  a.src = static_cast<const uint16_t*>(gu);
  a.src_ld = 2 * F;
  if ((st = fused<kEpiGluBwd>(h, ph, a, hs, dgus, s)) != GEMM_OK) return st;
  // dw_down [D, F] = dy^T h; dx = dg Wg + du Wu (two segments); the halves of
  // dw_in, dg^T x and du^T x (a batch of two).
  const Product pd = {D, F, T, dys, hs, true, true, bf16, 1, 1};
  if ((st = product(h, pd, {dw_down, D, F, F, 1, D * F}, kEarlyA, s)) != GEMM_OK) return st;
  const Product px = {T, D, F, dgus, w_ins, false, true, bf16, 1, 2, 0, 0, 0, {0, 1, 0}, {0, 1, 0}};
  if ((st = product(h, px, {dx, T, D, lddx, 1, T * lddx}, kEarlyA | kEarlyB, s)) != GEMM_OK) return st;
  const Product pi = {F, D, T, dgus, {x, T, D, ldx, 1, T * ldx}, true, true, bf16, 2, 1, 1, 0, 1};
  return product(h, pi, {dw_in, F, D, D, 2, F * D}, kEarlyA | kEarlyB, s);
}

size_t gemm_w4_workspace(gemm_ops_t h, int64_t T, int64_t N, int64_t K, int32_t gated) {
  return gated ? w4_workspace<true>(h, T, N, K) : w4_workspace<false>(h, T, N, K);
}

static gemm_status_t w4_run(gemm_ops_t h, const void* x, int64_t ldx, const void* codes,
                            const void* scales, const void* zeros, void* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int64_t group,
                            gemm_act_t act, gemm_dtype_t dtype, bool gated, void* stream) {
  if (!h || !dim_ok(T) || !dim_ok(N) || !dim_ok(K) || N > INT32_MAX / 2 || T > kMaxW4Tokens)
    return GEMM_ERR_INVALID_ARG;
  if (act < GEMM_ACT_SILU || act > GEMM_ACT_RELU) return GEMM_ERR_INVALID_ARG;
  if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
  if (group < 32 || group > (1 << 30) || (group & (group - 1)) != 0 || K % group != 0)
    return GEMM_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return GEMM_OK;
  if (ldy < N || K / 2 > kMaxStreamRow) return GEMM_ERR_INVALID_ARG;
  gemm_status_t st = check_ld(ldx, K);
  if (st != GEMM_OK) return st;
  if (!aligned16(x) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 1) ||
      (reinterpret_cast<uintptr_t>(y) & 1))
    return GEMM_ERR_ALIGNMENT;
  const size_t need = gemm_w4_workspace(h, T, N, K, gated);
  if (workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return GEMM_ERR_ALIGNMENT;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const int64_t rows = gated ? 2 * N : N, groups = K / group;
  const Buf bufs[] = {{x, T, K * 2, ldx * 2, false},
                      {codes, rows, K / 2, K / 2, false},
                      {scales, rows, groups * 2, groups * 2, false},
                      {zeros, zeros ? rows : 0, groups, groups, false},
                      {y, T, N * 2, ldy * 2, true},
                      {workspace, need ? 1 : 0, static_cast<int64_t>(need), 0, true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return cudaMemset2DAsync(y, ldy * 2, 0, N * 2, T, s) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  int shift = 0;
  while ((1ll << shift) < group) ++shift;
  StreamArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.w = codes;
  a.ldw = K / 2;
  a.scales = static_cast<const uint16_t*>(scales);
  a.zeros = static_cast<const uint8_t*>(zeros);
  a.y = static_cast<uint16_t*>(y);
  a.ldy = ldy;
  a.partial = static_cast<float*>(workspace);
  a.T = static_cast<int32_t>(T);
  a.K = static_cast<int32_t>(K);
  a.cols = static_cast<int32_t>(N);
  a.group_shift = shift;
  a.act = act;
  const bool bf16 = dtype == GEMM_BF16;
  return gated ? w4_product<true>(h, a, group, bf16, s) : w4_product<false>(h, a, group, bf16, s);
}

gemm_status_t gemm_w4_linear(gemm_ops_t h, const void* x, int64_t ldx, const void* codes,
                             const void* scales, const void* zeros, void* y, int64_t ldy, void* workspace,
                             size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int64_t group,
                             gemm_dtype_t dtype, void* stream) {
  return w4_run(h, x, ldx, codes, scales, zeros, y, ldy, workspace, workspace_bytes, T, N, K, group,
                GEMM_ACT_SILU, dtype, false, stream);
}

gemm_status_t gemm_w4_gated(gemm_ops_t h, const void* x, int64_t ldx, const void* codes,
                            const void* scales, const void* zeros, void* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, int64_t T, int64_t N, int64_t K, int64_t group,
                            gemm_act_t act, gemm_dtype_t dtype, void* stream) {
  return w4_run(h, x, ldx, codes, scales, zeros, y, ldy, workspace, workspace_bytes, T, N, K, group, act, dtype,
                true, stream);
}

size_t gemm_orthogonalize_workspace(gemm_ops_t h, int64_t batch, int64_t M, int64_t N) {
  if (!h || batch <= 0 || M <= 0 || N <= 0 || batch > 65535 || !dim_ok(M) || !dim_ok(N)) return 0;
  return ortho_space(batch, M, N).total;
}

gemm_status_t gemm_orthogonalize(gemm_ops_t h, const void* m, int64_t ldm, int64_t stride_m, void* out,
                                 int64_t ldo, int64_t stride_o, void* workspace, size_t workspace_bytes,
                                 int64_t batch, int64_t M, int64_t N, int32_t steps,
                                 const float coeffs[3], float eps, gemm_dtype_t in_dtype,
                                 gemm_dtype_t out_dtype, void* stream) {
  if (!h || !coeffs || !dim_ok(batch) || !dim_ok(M) || !dim_ok(N) || batch > 65535 || steps < 0)
    return GEMM_ERR_INVALID_ARG;
  for (gemm_dtype_t d : {in_dtype, out_dtype})
    if (d != GEMM_F16 && d != GEMM_BF16 && d != GEMM_F32) return GEMM_ERR_INVALID_ARG;
  if (!(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  if (batch == 0 || M == 0 || N == 0) return GEMM_OK;
  if (ldm < N || ldo < N || (batch > 1 && (stride_m < 0 || stride_o < (M - 1) * ldo + N)))
    return GEMM_ERR_INVALID_ARG;
  const int64_t ei = in_dtype == GEMM_F32 ? 4 : 2, eo = out_dtype == GEMM_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(m) % ei) || (reinterpret_cast<uintptr_t>(out) % eo) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GEMM_ERR_ALIGNMENT;
  const OrthoSpace sp = ortho_space(batch, M, N);
  if (workspace_bytes < sp.total) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const Buf bufs[] = {{m, M, N * ei, ldm * ei, false, batch, batch > 1 ? stride_m * ei : 0},
                      {out, M, N * eo, ldo * eo, true, batch, batch > 1 ? stride_o * eo : 0},
                      {workspace, 1, static_cast<int64_t>(sp.total), 0, true}};
  gemm_status_t st = check_bufs(h, bufs);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // X, P and Q = b P + c P^2 are held scaled by these powers of two.
  constexpr float kSx = 8192.0f, kSp = 2048.0f, kSq = 1024.0f;
  char* ws = static_cast<char*>(workspace);
  uint16_t* x[2] = {reinterpret_cast<uint16_t*>(ws + sp.x0), reinterpret_cast<uint16_t*>(ws + sp.x1)};
  uint16_t* P = reinterpret_cast<uint16_t*>(ws + sp.p);
  uint16_t* Q = reinterpret_cast<uint16_t*>(ws + sp.q);
  OrthoArgs oa = {};
  oa.in = m;
  oa.ld = ldm;
  oa.bs = batch > 1 ? stride_m : 0;
  oa.dtype = in_dtype;
  oa.rows = static_cast<int32_t>(M);
  oa.cols = static_cast<int32_t>(N);
  oa.x = x[0];
  oa.pitch = sp.pitch;
  oa.partial = reinterpret_cast<float*>(ws + sp.partial);
  oa.eps = eps;
  oa.scale = kSx;
  const unsigned by = static_cast<unsigned>(batch);
  if ((st = launch(h, ortho_norm, dim3(kNormBlocks, by), dim3(256), 0, 1, s, oa)) != GEMM_OK) return st;
  const unsigned bx = static_cast<unsigned>(std::min<int64_t>(M, cdiv(8 * h->num_sms, batch)));
  if ((st = launch(h, ortho_split, dim3(bx, by), dim3(256), 0, 1, s, oa)) != GEMM_OK) return st;
  const bool wide = M <= N;
  const int64_t r = sp.r, xpart = M * sp.pitch, ppart = r * sp.pitch_r;
  const float ca = coeffs[0], cb = coeffs[1], cc = coeffs[2];
  const Stack ps = {P, r, r, sp.pitch_r, 2 * batch, ppart}, qs = {Q, r, r, sp.pitch_r, 2 * batch, ppart};
  int cur = 0;
  for (int i = 0; i < steps; ++i, cur ^= 1) {
    const Stack xs = {x[cur], M, N, sp.pitch, 2 * batch, xpart};
    const Stack xn = {x[cur ^ 1], M, N, sp.pitch, 2 * batch, xpart};
    {  // P = X X^T (X^T X)
      const Product p = {r, r, wide ? N : M, xs, xs, !wide, !wide, false, batch, 3, 2, 2, 2, {0, 0, 1}, {0, 1, 0}};
      FusedArgs a = base_args(h, p);
      a.alpha = kSp / (kSx * kSx);
      if ((st = fused<kEpiSplitSym>(h, p, a, ps, ps, s)) != GEMM_OK) return st;
    }
    {  // Q = c P P + b P
      const Product p = {r, r, r, ps, ps, false, false, false, batch, 3, 2, 2, 2, {0, 0, 1}, {0, 1, 0}};
      FusedArgs a = base_args(h, p);
      a.alpha = cc * (kSq / (kSp * kSp));
      a.beta = cb * (kSq / kSp);
      a.src = P;
      a.src_ld = sp.pitch_r;
      a.src_part = ppart;
      if ((st = fused<kEpiSplitSym>(h, p, a, qs, qs, s)) != GEMM_OK) return st;
    }
    {  // X <- Q X + a X (X Q + a X); Q is symmetric
      const Product p = wide ? Product{M, N, r, qs, xs, false, true, false, batch, 3, 2, 2, 2, {0, 0, 1}, {0, 1, 0}}
                             : Product{M, N, r, xs, qs, false, false, false, batch, 3, 2, 2, 2, {0, 0, 1}, {0, 1, 0}};
      FusedArgs a = base_args(h, p);
      a.alpha = 1.0f / kSq;
      a.beta = ca;
      a.src = x[cur];
      a.src_ld = sp.pitch;
      a.src_part = xpart;
      if ((st = fused<kEpiSplit>(h, p, a, xn, {}, s)) != GEMM_OK) return st;
    }
  }
  oa.x = x[cur];
  oa.dtype = out_dtype;
  oa.out = out;
  oa.ld_out = ldo;
  oa.bs_out = batch > 1 ? stride_o : 0;
  return launch(h, ortho_join, dim3(bx, by), dim3(256), 0, 1, s, oa);
}

}  // extern "C"
