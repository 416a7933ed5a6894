// xent.cu -- host side of the vocabulary's loss and its gradients.
#include "host.cuh"
#include "xent_kernels.cuh"

namespace gb300 {
namespace ops {

bool xent_setup(gemm_ops_s* h) {
  if (!set_attr<WideLse>() || !set_attr<Pair<kEpiLse>>() || !set_attr<Lone<kEpiLse>>() || !set_attr<Lone<kEpiLse, 2>>() ||
      !set_attr<Lone<kEpiLse, 4>>() || !set_attr<Lone<kEpiLse, 8>>() || !set_attr<Pair<kEpiXent>>() ||
      !set_attr<Lone<kEpiXent>>() || !set_attr<Lone<kEpiXent, 2>>() || !set_attr<Lone<kEpiXent, 4>>() ||
      !set_attr<Lone<kEpiXent, 8>>() || !set_attr<Pair<kEpiSum>>() || !set_attr<Lone<kEpiSum>>() ||
      !set_attr<Long<Pair<kEpiSum>>>() || !set_attr<Long<Lone<kEpiSum>>>() || !set_attr<Long<Pair<kEpiStoreLive>>>() ||
      !set_attr<Long<Lone<kEpiStoreLive>>>() || !set_attr<Pair<kEpiStoreLive>>() || !set_attr<TwoPairs<kEpiStoreLive>>() || !set_attr<Lone<kEpiStoreLive>>() ||
      !set_attr<Lone<kEpiStoreLive, 2>>() || !set_attr<Lone<kEpiStoreLive, 4>>() || !set_attr<Lone<kEpiStoreLive, 8>>())
    return false;
  if (!set_attr<Long<Lone<kEpiLse, 2>>>() || !set_attr<Long<Lone<kEpiLse, 4>>>() || !set_attr<Long<Lone<kEpiLse, 8>>>() ||
      !set_attr<Long<Lone<kEpiXent, 2>>>() || !set_attr<Long<Lone<kEpiXent, 4>>>() || !set_attr<Long<Lone<kEpiXent, 8>>>())
    return false;
  h->max_pairs = std::min({h->max_pairs, max_clusters<Pair<kEpiLse>>(), max_clusters<Pair<kEpiXent>>(),
                           max_clusters<Pair<kEpiSum>>(), max_clusters<Pair<kEpiStoreLive>>(),
                           max_clusters<Long<Pair<kEpiSum>>>(), max_clusters<Long<Pair<kEpiStoreLive>>>()});
  h->max_twos = std::min(h->max_twos, max_clusters<TwoPairs<kEpiStoreLive>>());
  return true;
}

}  // namespace ops
}  // namespace gb300

namespace {

using namespace gb300::ops;

// Tokens of one launch of the forward pass at most, and bytes of their shares.
constexpr int64_t kLseTokens = 16384, kShareBytes = 512ll << 20;
// Bytes of dz held at a time, where pieces of kMinPiece columns allow it.
constexpr int64_t kPieceBytes = 512ll << 20, kMinPiece = 4096;
constexpr int64_t kMaxVocab = 1 << 28, kMaxWidth = 1 << 24;

bool xent_dims_ok(int64_t T, int64_t D, int64_t V) {
  return dim_ok(T) && D > 0 && D <= kMaxWidth && V > 0 && V <= kMaxVocab;
}

gemm_status_t check_xent(const gemm_ops_s* h, int64_t T, int64_t D, int64_t V, gemm_dtype_t dtype) {
  if (!h || !xent_dims_ok(T, D, V)) return GEMM_ERR_INVALID_ARG;
  if (dtype != GEMM_F16 && dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
  return D % 8 != 0 ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

// The most shares that any form leaves: one of 64 columns, four of a pair's tile, or
// sixteen of one of at most 76 tiles that a cluster shares.
int64_t most_shares(int64_t V) { return std::max<int64_t>(4 * cdiv(V, 256), std::min<int64_t>(16 * cdiv(V, 128), 16 * 76)); }

// Tokens of a launch: a multiple of a pair's 256 rows.
int64_t lse_tokens(int64_t T, int64_t V) {
  return std::min(T, std::clamp<int64_t>(kShareBytes / (8 * most_shares(V)) / 256 * 256, 256, kLseTokens));
}
size_t target_bytes(int64_t n) { return up(n * 4, 256); }

// Whether the forward pass copies x to rows in whole 128-byte lines: rows that straddle
// them are loaded as such for every tile of columns.  Without and with the copy: 500 x
// 1032 x 20011 29.7 and 28.0 us, 2598 x 3112 x 1161 29.5 and 27.6, 801 x 3160 x 60288
// 276 and 237, 3708 x 1880 x 58569 570 and 517.  Few rows are one tile anyway.
bool copies_x(int64_t T, int64_t D, int64_t V) { return D % 64 != 0 && T >= 256 && T * V >= 1 << 21; }

// Tile rows of logits that are worked on before the next columns of W: as many as 32 MB of
// x hold, which stay in L2 while W streams past them (eight, and by this rule: 16384 x
// 1024 x 32768 630 and 609 us, its gradients 2060 and 2010, of 8192 x 2048 x 65536 4150
// and 4030).
int32_t logits_group(int64_t D) { return static_cast<int32_t>(std::clamp<int64_t>((32 << 20) / (512 * D), kGroupM, 32)); }

// Columns of a piece of the vocabulary: as few equal pieces as fit.
int64_t piece_columns(int64_t T, int64_t V) {
  const int64_t most = std::max(kMinPiece, kPieceBytes / (2 * T) / 256 * 256);
  return V <= most ? V : up(cdiv(V, cdiv(V, most)), 256);
}

// Shares of the k-blocks (64 entries of the vocabulary) that are summed on their own for
// dx of few tiles, 0 where the forms that finish dx at once take no longer by the model in
// host.cuh: as many as lone CTAs or pairs run at once.  Writing the shares and adding them
// up takes 4 us.  4 x 1288 x 66557 148 us with clusters of four, 121 with 13 shares.
constexpr int64_t kAddShares = 400;
int64_t dx_slices(const gemm_ops_s* h, int64_t T, int64_t D, int64_t V) {
  const int64_t kb = cdiv(V, 64);
  int64_t slices = 0, least = form_costs<kEpiStoreLive>(h, T, D, kb, 1, true).least();
  for (int64_t fit : {h->num_sms / (cdiv(T, 128) * cdiv(D, 128)), h->max_pairs / (cdiv(T, 256) * cdiv(D, 256))}) {
    const int64_t s = std::min(fit, kb / 8);
    if (s < 2) continue;
    const int64_t cost = form_costs<kEpiSum>(h, T, D, cdiv(kb, s), s, false).least() + kAddShares;
    if (cost < least) least = cost, slices = s;
  }
  return slices;
}

struct XentSpace {
  int64_t piece, pitch, pitch_x, slices;  // pitch_x: of the copy of x, in whole 128-byte lines
  size_t rows, scalars, order, packed, dz, sum, total;
};
XentSpace xent_space(const gemm_ops_s* h, int64_t T, int64_t D, int64_t V) {
  XentSpace s;
  s.piece = piece_columns(T, V);
  s.pitch = up(s.piece, 64);
  s.pitch_x = up(D, 64);
  s.rows = 0;
  s.scalars = up(T * static_cast<int64_t>(sizeof(XentRow)), 256);
  s.order = s.scalars + 256;
  s.packed = s.order + up(T * 4, 256);
  s.dz = s.packed + up(T * s.pitch_x * 2, 256);
  s.sum = s.dz + up(T * s.pitch * 2, 256);
  // Several pieces, or shares of one: fp32 sums of dx.
  s.slices = s.piece < V ? 1 : dx_slices(h, T, D, V);
  s.total = s.sum + up(s.slices * T * D * 4, 256);
  return s;
}

}  // namespace

extern "C" {

size_t gemm_linear_cross_entropy_workspace(gemm_ops_t h, int64_t T, int64_t D, int64_t V) {
  if (!h || T <= 0 || !xent_dims_ok(T, D, V)) return 0;
  const int64_t n = lse_tokens(T, V);
  return target_bytes(n) + up(most_shares(V) * n * 8, 256) + (copies_x(T, D, V) ? up(n * up(D, 64) * 2, 256) : 0);
}

gemm_status_t gemm_linear_cross_entropy(gemm_ops_t h, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                        const int64_t* targets, float* loss, float* lse, void* workspace,
                                        size_t workspace_bytes, int64_t T, int64_t D, int64_t V,
                                        int64_t ignore_index, gemm_dtype_t dtype, void* stream) {
  gemm_status_t st = check_xent(h, T, D, V, dtype);
  if (st != GEMM_OK) return st;
  if (T == 0) return GEMM_OK;
  for (auto ld : {ldx, ldw})
    if ((st = check_ld(ld, D)) != GEMM_OK) return st;
  if (!aligned16(x) || !aligned16(w) || (reinterpret_cast<uintptr_t>(targets) & 7) ||
      (reinterpret_cast<uintptr_t>(loss) & 3) || (reinterpret_cast<uintptr_t>(lse) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GEMM_ERR_ALIGNMENT;
  const size_t need = gemm_linear_cross_entropy_workspace(h, T, D, V);
  if (workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const Buf bufs[] = {{x, T, D * 2, ldx * 2, false},
                      {w, V, D * 2, ldw * 2, false},
                      {targets, T, 8, 8, false},
                      {loss, T, 4, 4, true},
                      {lse, lse ? T : 0, 4, 4, true},
                      {workspace, 1, static_cast<int64_t>(need), static_cast<int64_t>(need), true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* target_z = static_cast<float*>(workspace);
  const int64_t step = lse_tokens(T, V);
  float2* shares = reinterpret_cast<float2*>(static_cast<char*>(workspace) + target_bytes(step));
  const bool copy = copies_x(T, D, V);
  void* packed = reinterpret_cast<char*>(shares) + up(most_shares(V) * step * 8, 256);
  for (int64_t t0 = 0; t0 < T; t0 += step) {
    const int64_t n = std::min(step, T - t0);
    XentArgs j = {};
    j.x = static_cast<const uint16_t*>(x) + t0 * ldx;
    j.ldx = ldx, j.D = D, j.T = n;
    j.packed = packed, j.pitch = up(D, 64);
    if (copy) {
      const int64_t blocks = std::min<int64_t>(cdiv(n * cdiv(D, 1024), 8), 8 * h->num_sms);
      if ((st = launch(h, xent_copy, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, 1, s, j)) != GEMM_OK) return st;
    }
    const Stack xs = copy ? Stack{packed, n, D, j.pitch, 1, n * j.pitch} : Stack{j.x, n, D, ldx, 1, n * ldx};
    const Product p = {n, V, D, xs, {w, V, D, ldw, 1, V * ldw}, false, false, dtype == GEMM_BF16, 1, 1};
    FusedArgs a = base_args(h, p);
    if (copy)
      a.early = kEarlyB;
    else if (t0 > 0)
      a.early = kEarlyA | kEarlyB;  // the kernels before wrote neither x nor W
    a.group_m = logits_group(D);
    a.targets = targets + t0;
    a.target_z = target_z;
    a.shares = shares;
    int64_t num = 0;
    if ((st = fused<kEpiLse>(h, p, a, {}, {}, s, &num)) != GEMM_OK) return st;
    j.targets = targets + t0;
    j.V = V, j.ignore = ignore_index;
    j.shares = shares, j.num_shares = num, j.target_z = target_z;
    j.loss = loss + t0, j.lse = lse ? lse + t0 : nullptr;
    int32_t per = 1;  // a block's tokens: 32 bytes of their shares at least, where there are as many
    while (per < 32 && per < n && (per < 4 || n / per > 2 * h->num_sms)) per *= 2;
    st = launch(h, xent_join, dim3(static_cast<unsigned>(cdiv(n, per))), dim3(kJoinThreads), 0, 1, s, j, per);
    if (st != GEMM_OK) return st;
  }
  return GEMM_OK;
}

size_t gemm_linear_cross_entropy_backward_workspace(gemm_ops_t h, int64_t T, int64_t D, int64_t V) {
  if (!h || T <= 0 || !xent_dims_ok(T, D, V)) return 0;
  return xent_space(h, T, D, V).total;
}

gemm_status_t gemm_linear_cross_entropy_backward(gemm_ops_t h, const float* dloss, int64_t dloss_stride,
                                                 const float* dlse, int64_t dlse_stride, const void* x, int64_t ldx,
                                                 const void* w, int64_t ldw, const int64_t* targets, const float* lse,
                                                 void* dx, int64_t lddx, void* dw, void* workspace,
                                                 size_t workspace_bytes, int64_t T, int64_t D, int64_t V,
                                                 int64_t ignore_index, gemm_dtype_t dtype, void* stream) {
  gemm_status_t st = check_xent(h, T, D, V, dtype);
  if (st != GEMM_OK) return st;
  if (dloss_stride < 0 || dlse_stride < 0 || dloss_stride >= (1ll << 30) || dlse_stride >= (1ll << 30))
    return GEMM_ERR_INVALID_ARG;
  for (auto ld : {ldx, ldw, lddx})
    if ((st = check_ld(ld, D)) != GEMM_OK) return st;
  if (!aligned16(x) || !aligned16(w) || !aligned16(dx) || !aligned16(dw) || (reinterpret_cast<uintptr_t>(targets) & 7) ||
      (reinterpret_cast<uintptr_t>(dloss) & 3) || (reinterpret_cast<uintptr_t>(dlse) & 3) ||
      (reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GEMM_ERR_ALIGNMENT;
  const size_t need = gemm_linear_cross_entropy_backward_workspace(h, T, D, V);
  if (workspace_bytes < need) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const Buf bufs[] = {{dloss, T, 4, dloss_stride * 4, false},
                      {dlse, dlse ? T : 0, 4, dlse_stride * 4, false},
                      {x, T, D * 2, ldx * 2, false},
                      {w, V, D * 2, ldw * 2, false},
                      {targets, T, 8, 8, false},
                      {lse, T, 4, 4, false},
                      {dx, T, D * 2, lddx * 2, true},
                      {dw, V, D * 2, D * 2, true},
                      {workspace, need ? 1 : 0, static_cast<int64_t>(need), static_cast<int64_t>(need), true}};
  if ((st = check_bufs(h, bufs)) != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)  // no token, no gradient
    return cudaMemsetAsync(dw, 0, V * D * 2, s) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  const bool bf16 = dtype == GEMM_BF16;
  const XentSpace sp = xent_space(h, T, D, V);
  char* ws = static_cast<char*>(workspace);
  XentArgs r = {};
  r.targets = targets;
  r.T = T, r.V = V, r.D = D, r.ignore = ignore_index;
  r.lse = const_cast<float*>(lse);
  r.dloss = dloss, r.dlse = dlse, r.dloss_stride = dloss_stride, r.dlse_stride = dlse_stride;
  r.x = x, r.ldx = ldx, r.dx = dx, r.lddx = lddx, r.bf16 = bf16;
  r.rows = reinterpret_cast<XentRow*>(ws + sp.rows);
  r.scale = reinterpret_cast<float*>(ws + sp.scalars);
  r.live = reinterpret_cast<int32_t*>(ws + sp.scalars) + 1;
  r.order = reinterpret_cast<int32_t*>(ws + sp.order);
  r.packed = ws + sp.packed;
  r.pitch = sp.pitch_x;
  r.hold = bf16 ? 1.0f : 16384.0f;
  r.sum = reinterpret_cast<const float*>(ws + sp.sum);
  r.slices = sp.slices;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(cdiv(T, 4), 2 * h->num_sms));
  if ((st = launch(h, xent_pack, dim3(blocks), dim3(kPackThreads), 0, 1, s, r)) != GEMM_OK) return st;
  void* dz = ws + sp.dz;
  const bool whole = sp.piece >= V;
  // Laid out for all T tokens; r.live of them take part.
  const Stack xs = {r.packed, T, D, sp.pitch_x, 1, T * sp.pitch_x};
  for (int64_t v0 = 0; v0 < V; v0 += sp.piece) {
    const int64_t n = std::min(sp.piece, V - v0);
    const Stack wv = {static_cast<const uint16_t*>(w) + v0 * ldw, n, D, ldw, 1, n * ldw};
    const Stack dzs = {dz, T, n, sp.pitch, 1, T * sp.pitch};
    {  // dz, from the logits x W^T: at least one tile, of zeros, for dW
      const Product p = {T, n, D, xs, wv, false, false, bf16, 1, 1};
      FusedArgs a = base_args(h, p);
      // (The first needs `live`, which the kernel before it writes, to know its tiles at all.)
      if (v0 > 0) a.early = kEarlyA | kEarlyB | kEarlyLive;
      a.live = r.live;
      a.live_min = 1;
      a.group_m = logits_group(D);
      a.xent_rows = r.rows;
      a.col_base = static_cast<int32_t>(v0);
      if ((st = fused<kEpiXent>(h, p, a, dzs, {}, s)) != GEMM_OK) return st;
    }
    {  // dx = dz W, right after dz, while W is in L2; or its sums over the pieces, or shares
      const Product p = {T, D, n, dzs, wv, false, true, bf16, std::max<int64_t>(1, whole ? sp.slices : 1), 1};
      FusedArgs a = base_args(h, p);
      a.early = kEarlyB | kEarlyLive;
      a.live = r.live;
      if (sp.slices == 0) {
        a.alpha_p = r.scale;
        a.row_map = r.order;
        st = fused<kEpiStoreLive>(h, p, a, {dx, T, D, lddx, 1, T * lddx}, {}, s);
      } else if (whole) {
        a.k_slices = static_cast<int32_t>(sp.slices);
        a.c_zb = 1;
        st = fused<kEpiSum>(h, p, a, {r.sum, T, D, D, sp.slices, T * D}, {}, s);
      } else {
        a.add = v0 > 0;
        st = fused<kEpiSum>(h, p, a, {r.sum, T, D, D, 1, T * D}, {}, s);
      }
      if (st != GEMM_OK) return st;
    }
    // dW = dz^T x, whole for this piece
    const Product p = {n, D, T, dzs, xs, true, true, bf16, 1, 1};
    FusedArgs a = base_args(h, p);
    a.early = kEarlyA | kEarlyB | kEarlyLive;
    a.live = r.live;
    a.live_k = 1;
    a.alpha_p = r.scale;
    const Stack out = {static_cast<uint16_t*>(dw) + v0 * D, n, D, D, 1, n * D};
    if ((st = fused<kEpiStoreLive>(h, p, a, out, {}, s)) != GEMM_OK) return st;
  }
  if (sp.slices == 0) return GEMM_OK;
  const int64_t ctas = std::min<int64_t>(cdiv(T * (D / 8), 256), 8 * h->num_sms);
  return launch(h, xent_dx, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, 1, s, r);
}

}  // extern "C"
