// host.cuh -- what the host sides of the operators share: the handle, checks of
// arguments, tensor maps, launches, and the choice of a fused product's form.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "fused_kernel.cuh"
#include "gemm_ops.h"

struct gemm_ops_s {
  int device = 0;
  int num_sms = 0;
  int max_pairs = 0;      // CTA pairs of the pair kernels that fit on the device at once
  int max_twos = 0;       // clusters of two pairs sharing a tile
  int max_split[4] = {};  // clusters of 1, 2, 4, 8 CTAs sharing a tile
  void* encode = nullptr;
  uint32_t* d_err = nullptr;  // 4-word watchdog record
  uint32_t last_err[4] = {0, 0, 0, 0};
  uint64_t timeout_ns = 2000000000ull;
  int32_t skip_kb = -1;
  std::atomic<uint64_t> launches{0};
};

namespace gb300 {
namespace ops {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int kGroupM = 8;

// Staging buffers of an epilogue warp: 64 KB in all beside five stages.
constexpr int epi_bufs(int epi) { return epi == kEpiSplit || epi == kEpiSplitSym ? 4 : 2; }

// Tile configurations: a pair of CTAs on 256 x 256 sums, or one CTA on
// 128 x 128 for problems of few tiles.
template <int kEpi>
using Pair = FusedCfg<2, 256, kEpi == kEpiLse ? 7 : kEpi == kEpiStore ? 6 : 5, kEpi,
                      kEpi == kEpiLse ? 0 : kEpi == kEpiStore || kEpi == kEpiXent ? 1 : epi_bufs(kEpi)>;
template <int kEpi>
using TwoPairs = FusedCfg<2, 256, 5, kEpi, epi_bufs(kEpi), 2, kEpi == kEpiStoreLive ? 2 : 1>;  // one tile, half of its k-blocks each
template <int kEpi, int kSplit = 1, int kParts = 1>
using Lone = FusedCfg<1, 128, kEpi == kEpiLse && kSplit == 1 ? 7 : 5, kEpi,
                      kEpi == kEpiLse && kSplit == 1 ? 0 : epi_bufs(kEpi), kSplit,
                      ((kEpi == kEpiLse || kEpi == kEpiXent || kEpi == kEpiStoreLive) && kSplit > 1) ? 4 : kParts>;

// dx and dW of long sums, clusters' logits of wide rows.
template <class Cfg>
using Long = FusedCfg<Cfg::kCtas, Cfg::kBN, Cfg::kStages, Cfg::kEpi, Cfg::kEpiBufs, Cfg::kSplit, 0>;

// One CTA on 128 x 256 logits of the loss, for the rounds that tiles of a pair or of 128
// columns fill badly: 1 token, 4096 x 32000 49.5 -> 45.1 us, 101 x 512 x 32000 13.4 ->
// 9.7, 333 x 1024 x 100003 79.6 -> 65.4.  (The backward pass's, with dz to stage and
// three k-blocks in flight, gained nothing.)
using WideLse = FusedCfg<1, 256, 4, kEpiLse, 0>;

struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) return;
    ok = (prev == dev) || (cudaSetDevice(dev) == cudaSuccess);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

inline bool on_device(const void* ptr, int dev) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, ptr) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice && at.device == dev;
}

// A buffer of a call: [rows] rows of `row` bytes, `pitch` bytes apart, in `batch`
// matrices `stride` bytes apart.
struct Buf {
  const void* p;
  int64_t rows, row, pitch;
  bool out;
  int64_t batch = 1, stride = 0;
  int64_t matrix() const { return (rows - 1) * pitch + row; }
  size_t bytes() const {
    return rows > 0 && row > 0 && batch > 0 ? static_cast<size_t>((batch - 1) * stride + matrix()) : 0;
  }
  uintptr_t at() const { return reinterpret_cast<uintptr_t>(p); }
};

// Whether units of x and y (wx and wy bytes, nx and ny of them, px and py apart)
// interleave without touching, as the halves of one matrix's columns do.  Units of
// one pitch only: a lone one takes the other's.
inline bool interleaved(uintptr_t x, int64_t wx, int64_t px, int64_t nx, uintptr_t y, int64_t wy, int64_t py, int64_t ny) {
  const int64_t p = nx > 1 ? px : py;
  if ((nx > 1 && ny > 1 && px != py) || p <= 0) return false;
  const int64_t d = static_cast<int64_t>((x % p + p - y % p) % p);  // of x's units behind y's
  return d >= wy && d + wx <= p;
}

inline bool overlap(const Buf& a, const Buf& b) {
  if (a.at() >= b.at() + b.bytes() || b.at() >= a.at() + a.bytes()) return false;
  // Whole matrices in turn, or rows, where every matrix starts on the same column.
  if (interleaved(a.at(), a.matrix(), a.stride, a.batch, b.at(), b.matrix(), b.stride, b.batch)) return false;
  const bool same = (a.batch <= 1 || (a.pitch > 0 && a.stride % a.pitch == 0)) &&
                    (b.batch <= 1 || (b.pitch > 0 && b.stride % b.pitch == 0));
  return !same || !interleaved(a.at(), a.row, a.pitch, a.rows * a.batch, b.at(), b.row, b.pitch, b.rows * b.batch);
}

// Device memory throughout, and no output overlapping another buffer.
template <int kN>
gemm_status_t check_bufs(const gemm_ops_s* h, const Buf (&b)[kN]) {
  for (int i = 0; i < kN; ++i) {
    if (b[i].bytes() == 0) continue;
    if (!b[i].p || !on_device(b[i].p, h->device)) return GEMM_ERR_INVALID_ARG;
    if (!b[i].out) continue;
    for (int j = 0; j < kN; ++j)
      if (j != i && b[j].bytes() != 0 && !(b[j].out && j < i) && overlap(b[i], b[j])) return GEMM_ERR_INVALID_ARG;
  }
  return GEMM_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// The kernels' 32-bit counters of rows and columns run past the end of a matrix
// by less than a tile (256 and 192 columns more), or by the stride of a loop: 256
// columns, or the rows of one round of CTAs, 8 per SM.
constexpr int64_t kMaxLength = INT32_MAX - 4095;
inline bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxLength; }
inline int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t cdiv(int64_t v, int64_t m) { return (v + m - 1) / m; }

// ------------------------------------------------------------ tensor maps --
// A stack of `z` row-major matrices of rows x cols, rows `pitch` and matrices
// `zstride` elements apart.
struct Stack {
  const void* p;
  int64_t rows, cols, pitch, z, zstride;
};

inline bool make_map(const gemm_ops_s* h, CUtensorMap* m, const Stack& s, gemm_dtype_t type, uint32_t box_cols,
                     uint32_t box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint64_t size = type == GEMM_F32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(s.cols), static_cast<cuuint64_t>(s.rows),
                              static_cast<cuuint64_t>(s.z)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s.pitch) * size,
                                 static_cast<cuuint64_t>(s.zstride) * size};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  // Rows whose pitch is not a multiple of 128 bytes straddle L2 lines:
  // promoting their requests to 256 bytes costs more than it saves.
  const CUtensorMapL2promotion l2 = s.pitch % 64 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  auto encode = [&] {
    return reinterpret_cast<EncodeTiledFn>(h->encode)(
        m,
        type == GEMM_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
        : type == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
        3, const_cast<void*>(s.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
        l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  // A host thread that has not used CUDA (autograd's, a worker's) has a device but
  // no context, which the driver's encoder needs: cudaSetDevice makes the primary
  // one current.
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaSetDevice(h->device) == cudaSuccess) r = encode();
  return r == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- launches --
template <class... Params, class... Args>
gemm_status_t launch(gemm_ops_s* h, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                     int cluster, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  // Set-up may overlap the end of the previous kernel of the stream; every
  // kernel waits for it before touching global memory.
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  ++h->launches;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

// One product: acc[M, N] over segs x K, A and B stacks, their layouts.
struct Product {
  int64_t M, N, K;
  Stack a, b;
  bool a_mn, b_mn;  // stored [K, M] / [K, N]
  bool bf16;
  int64_t batch, segs;
  int32_t a_zb, b_zb, c_zb;   // stack coordinates: FusedArgs
  int32_t a_seg[3], b_seg[3];
};

inline FusedArgs base_args(const gemm_ops_s* h, const Product& p) {
  FusedArgs a = {};
  a.M = static_cast<int32_t>(p.M);
  a.N = static_cast<int32_t>(p.N);
  a.num_kb = static_cast<int32_t>(cdiv(p.K, 64));
  a.segs = static_cast<int32_t>(p.segs);
  a.a_zb = p.a_zb;
  a.b_zb = p.b_zb;
  a.c_zb = p.c_zb;
  for (int i = 0; i < 3; ++i) {
    a.a_seg[i] = p.a_seg[i];
    a.b_seg[i] = p.b_seg[i];
  }
  a.group_m = kGroupM;
  a.a_mn = p.a_mn;
  a.b_mn = p.b_mn;
  a.bf16 = p.bf16;
  a.alpha = 1.0f;
  a.err = h->d_err;
  a.timeout_ns = h->timeout_ns;
  a.skip_kb = h->skip_kb;
  return a;
}

template <class Cfg>
gemm_status_t launch_fused(gemm_ops_s* h, const Product& p, FusedArgs a, const Stack& c,
                           const Stack& d, cudaStream_t stream, int64_t* shares = nullptr) {
  CUtensorMap ma, mb, mc, md;
  const uint32_t b_rows = Cfg::kGlu && Cfg::kCtas == 1 ? Cfg::kBN / 2 : Cfg::kBRows;
  // Fewer rows than a tile: a box of those alone, and more k-blocks in flight.
  // What the MMA takes for the tile's other rows, the bytes that follow, meets
  // no stored row of the product.  24 tokens, weights of 8192 x 16384 and of
  // 2048 x 5632: whole boxes 143.4 and 30.6 us, boxes of 24 rows 142.7 and
  // 25.7 us, with eight k-blocks in flight in place of five 133.8 and 25.4 us.
  const uint32_t a_rows =
      Cfg::kCtas == 1 && !p.a_mn ? static_cast<uint32_t>(std::min<int64_t>(Cfg::kBM, up(p.M, 8))) : Cfg::kBM;
  a.a_tx = a_rows * Cfg::kBK * 2;
  a.stages = std::min<int32_t>(Cfg::kMaxStages, Cfg::kStages * (Cfg::kABytes + Cfg::kBBytes) / (a.a_tx + Cfg::kBBytes));
  const gemm_dtype_t type = p.bf16 ? GEMM_BF16 : GEMM_F16;
  bool ok = make_map(h, &ma, p.a, type, 64, p.a_mn ? 64 : a_rows) &&
            make_map(h, &mb, p.b, type, 64, p.b_mn ? 64 : b_rows);
  if (ok && c.p)
    ok = Cfg::kEpi == kEpiSum ? make_map(h, &mc, c, GEMM_F32, 32, 32) : make_map(h, &mc, c, type, 64, 32);
  if (ok && d.p)
    ok = Cfg::kSym ? make_map(h, &md, d, type, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE)
                   : make_map(h, &md, d, type, 64, 32);
  if (!ok) return GEMM_ERR_CUDA;
  if (!c.p) mc = ma;  // not used by this epilogue
  if (!d.p) md = ma;
  const int64_t tm = cdiv(p.M, Cfg::kTileM), tn = cdiv(p.N, Cfg::kOutN);
  const int64_t per = Cfg::kSym ? tn * (tn + 1) / 2 : tm * tn;
  const int64_t items = per * p.batch;
  if (items > INT32_MAX / 2) return GEMM_ERR_INVALID_ARG;
  a.tiles_m = static_cast<int32_t>(tm);
  a.tiles_n = static_cast<int32_t>(tn);
  a.per_batch = static_cast<int32_t>(per);
  a.items = static_cast<int32_t>(items);
  a.c = static_cast<uint16_t*>(const_cast<void*>(c.p));
  a.ldc = c.pitch;
  a.c_z = c.zstride;
  a.ldd = d.pitch;
  a.d_up = d.zstride;
  a.d = static_cast<uint16_t*>(const_cast<void*>(d.p));
  if (shares) *shares = tn * (Cfg::kSplit > 1 ? 2 * Cfg::kSplit : Cfg::kGroups);  // kEpiLse
  const int64_t fit = Cfg::kCtas == 2 ? h->max_pairs : h->num_sms;
  const int64_t units = Cfg::kSplit > 1 ? items : std::min<int64_t>(items, fit);
  return launch(h, fused_kernel<Cfg>, dim3(static_cast<unsigned>(units * Cfg::kCluster)), dim3(Cfg::kThreads),
                Cfg::kSmemBytes, Cfg::kCluster, stream, ma, mb, mc, md, a);
}

// Which form: the one whose rounds of tiles take the least time by this model,
// in units of 10 ns: a k-block takes a lone CTA 0.27 us (its 32 KB of operands
// through the SM's L2 port; 0.4 us and 48 KB for 256 columns), a pair 0.33 us (the
// tensor pipe), and a tile starts and ends in 4 to 7 us.  Of clusters of two CTAs 76
// fit at once, of four 36, of eight 15.  Lone clusters split a tile only where all fit
// at once.
//
// The batched products (high and low parts) go by one matrix's tiles alone, so
// that a matrix of a batch gets the same sums as by itself: the number of its
// k-ranges is fixed, and the batch's tiles decide who sums them.
enum Form { kPairs, kPairs2, kLone, kLone2, kLone4, kLone8, kWide, kForms };
struct FormCosts {
  static constexpr int64_t kNever = INT64_MAX;
  int64_t small;  // tiles of lone CTAs
  int64_t cost[kForms];
  Form best() const { return static_cast<Form>(std::min_element(cost, cost + kForms) - cost); }
  int64_t least() const { return cost[best()]; }
};

// Whether matrices of a batch are to get the same sums as by themselves.
template <int kEpi>
constexpr bool kBatched = kEpi == kEpiSplit || kEpi == kEpiSplitSym;
// Which forms there are.  The loss's sums have tiles enough, or shares of the k-blocks.
template <int kEpi>
constexpr bool kSplits = kEpi != kEpiSum;
template <int kEpi>
constexpr bool kTwos = kSplits<kEpi> && kEpi != kEpiLse && kEpi != kEpiXent;

// Of M x N sums over kb k-blocks, n times.  may_split false: a k-range of fewer k-blocks
// than the launch was laid out for could be empty.
template <int kEpi>
FormCosts form_costs(const gemm_ops_s* h, int64_t M, int64_t N, int64_t kb, int64_t n, bool may_split) {
  constexpr int64_t kNever = FormCosts::kNever;
  const bool split = kSplits<kEpi> && may_split;
  auto tiles = [&](int64_t tm, int64_t tn) { return Pair<kEpi>::kSym ? tn * (tn + 1) / 2 : tm * tn; };
  const int64_t small = tiles(cdiv(M, 128), cdiv(N, Lone<kEpi>::kOutN)) * n;
  const int64_t big = tiles(cdiv(M, 256), cdiv(N, Pair<kEpi>::kOutN)) * n;
  const int64_t wide = cdiv(M, 128) * cdiv(N, 256);
  const int* most = h->max_split;
  // k-blocks that a cluster's CTA has room to sum: dx's four or (of pairs) two accumulators.
  const int64_t room = kEpi == kEpiStoreLive ? 4 * kSumKb : kNever / 8;
  const int64_t room_two = kEpi == kEpiStoreLive ? 2 * kSumKb : kNever / 8;
  FormCosts f = {small, {}};
  std::fill(f.cost, f.cost + kForms, kNever);
  if (h->max_pairs > 0) f.cost[kPairs] = cdiv(big, h->max_pairs) * (33 * kb + 500);
  if (kTwos<kEpi> && split && h->max_twos > 0 && kb >= 4 && kb <= 2 * room_two)
    f.cost[kPairs2] = cdiv(big, h->max_twos) * (33 * cdiv(kb, 2) + 700);
  f.cost[kLone] = cdiv(small, h->num_sms) * (27 * kb + 400);
  if (split && small <= most[1] && kb >= 4 && kb <= 2 * room) f.cost[kLone2] = 27 * cdiv(kb, 2) + 550;
  if (split && small <= most[2] && kb >= (kBatched<kEpi> ? 4 : 8) && kb <= 4 * room) f.cost[kLone4] = 27 * cdiv(kb, 4) + 550;
  if (split && !kBatched<kEpi> && small <= std::min(8, most[3]) && kb >= 16 && kb <= 8 * room)
    f.cost[kLone8] = 27 * cdiv(kb, 8) + 550;
  if (kEpi == kEpiLse) f.cost[kWide] = cdiv(wide, h->num_sms) * (40 * kb + 450);
  return f;
}

template <int kEpi>
gemm_status_t fused(gemm_ops_s* h, const Product& p, const FusedArgs& a, const Stack& c,
                    const Stack& d, cudaStream_t stream, int64_t* shares = nullptr) {
  const int64_t n = kBatched<kEpi> ? 1 : p.batch, kb = cdiv(cdiv(p.K, 64) * p.segs, std::max(1, a.k_slices));
  const FormCosts f = form_costs<kEpi>(h, p.M, p.N, kb, n, !(Pair<kEpi>::kLive && a.live_k));
  const Form form = f.best();
  if constexpr (Lone<kEpi>::kSums)
    if (kb > kSumKb) {
      if (form == kPairs) return launch_fused<Long<Pair<kEpi>>>(h, p, a, c, d, stream, shares);
      if (form == kLone) return launch_fused<Long<Lone<kEpi>>>(h, p, a, c, d, stream, shares);
    }
  switch (form) {
    case kPairs: return launch_fused<Pair<kEpi>>(h, p, a, c, d, stream, shares);
    case kPairs2:
      if constexpr (kTwos<kEpi>) return launch_fused<TwoPairs<kEpi>>(h, p, a, c, d, stream, shares);
      break;
    case kLone2:
      if constexpr (kBatched<kEpi>)
        if (f.small * p.batch > h->max_split[1]) return launch_fused<Lone<kEpi, 1, 2>>(h, p, a, c, d, stream, shares);
      if constexpr (Lone<kEpi>::kPartial)
        if (kb > 2 * 4 * kSplitKb) return launch_fused<Long<Lone<kEpi, 2>>>(h, p, a, c, d, stream, shares);
      if constexpr (kSplits<kEpi>) return launch_fused<Lone<kEpi, 2>>(h, p, a, c, d, stream, shares);
      break;
    case kLone4:
      if constexpr (kBatched<kEpi>)
        if (f.small * p.batch > h->max_split[2]) return launch_fused<Lone<kEpi, 1, 4>>(h, p, a, c, d, stream, shares);
      if constexpr (Lone<kEpi>::kPartial)
        if (kb > 4 * 4 * kSplitKb) return launch_fused<Long<Lone<kEpi, 4>>>(h, p, a, c, d, stream, shares);
      if constexpr (kSplits<kEpi>) return launch_fused<Lone<kEpi, 4>>(h, p, a, c, d, stream, shares);
      break;
    case kLone8:
      if constexpr (Lone<kEpi>::kPartial)
        if (kb > 8 * 4 * kSplitKb) return launch_fused<Long<Lone<kEpi, 8>>>(h, p, a, c, d, stream, shares);
      if constexpr (kSplits<kEpi> && !kBatched<kEpi>) return launch_fused<Lone<kEpi, 8>>(h, p, a, c, d, stream, shares);
      break;
    case kWide:
      if constexpr (kEpi == kEpiLse) return launch_fused<WideLse>(h, p, a, c, d, stream, shares);
      break;
    default: break;
  }
  return launch_fused<Lone<kEpi>>(h, p, a, c, d, stream, shares);
}

// `early`: operands (and FusedArgs::live) that may be loaded while the previous
// kernel ends.  A kernel of the operators lets the next one start only after it has
// waited for the one before it, so what is complete by then are the caller's tensors,
// and what the last kernel but one wrote.
enum { kEarlyA = 1, kEarlyB = 2, kEarlyLive = 4 };

// Attributes of the loss's kernels, and how many of their clusters fit.
bool xent_setup(gemm_ops_s* h);

template <class Cfg>
bool set_attr() {
  return cudaFuncSetAttribute(fused_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg::kSmemBytes) == cudaSuccess;
}

template <class Cfg>
int max_clusters() {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(Cfg::kCluster, 1, 1);
  cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = Cfg::kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fused_kernel<Cfg>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

inline gemm_status_t check_ld(int64_t ld, int64_t cols) {
  if (ld < cols || ld >= (1ll << 30)) return GEMM_ERR_INVALID_ARG;
  return ld % 8 != 0 ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

}  // namespace ops
}  // namespace gb300
