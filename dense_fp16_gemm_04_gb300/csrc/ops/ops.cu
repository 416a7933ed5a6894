// ops.cu -- host side of the C ABI declared in include/gemm_ops.h: argument
// checks, tensor maps, the choice of kernel and the launches.
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
#include "ortho_kernels.cuh"
#include "stream_kernel.cuh"

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

namespace {

using namespace gb300::ops;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
// Tokens of the streaming products of 16-bit weights; more go to the tensor
// cores' own products.  16 and 17 tokens: weights of 1024 x 4096 11.4 and 13.7
// us, 2048 x 5632 22.1 and 25.3 us, 4096 x 8192 46.3 and 41.7 us, 8192 x 16384
// 145 and 133 us.
constexpr int64_t kMaxStreamTokens = 16;
constexpr int kGroupM = 8;

// Staging buffers of an epilogue warp: 64 KB in all beside five stages.
constexpr int epi_bufs(int epi) { return epi == kEpiSplit || epi == kEpiSplitSym ? 4 : 2; }

// Tile configurations: a pair of CTAs on 256 x 256 sums, or one CTA on
// 128 x 128 for problems of few tiles.
template <int kEpi>
using Pair = FusedCfg<2, 256, kEpi == kEpiStore ? 6 : 5, kEpi, kEpi == kEpiStore ? 1 : epi_bufs(kEpi)>;
template <int kEpi>
using TwoPairs = FusedCfg<2, 256, 5, kEpi, epi_bufs(kEpi), 2>;  // one tile, half of its k-blocks each
template <int kEpi, int kSplit = 1, int kParts = 1>
using Lone = FusedCfg<1, 128, 5, kEpi, epi_bufs(kEpi), kSplit, kParts>;

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

bool on_device(const void* ptr, int dev) {
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
bool interleaved(uintptr_t x, int64_t wx, int64_t px, int64_t nx, uintptr_t y, int64_t wy, int64_t py, int64_t ny) {
  const int64_t p = nx > 1 ? px : py;
  if ((nx > 1 && ny > 1 && px != py) || p <= 0) return false;
  const int64_t d = static_cast<int64_t>((x % p + p - y % p) % p);  // of x's units behind y's
  return d >= wy && d + wx <= p;
}

bool overlap(const Buf& a, const Buf& b) {
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// The kernels' 32-bit counters of rows and columns run past the end of a matrix
// by less than a tile (256 and 192 columns more), or by the stride of a loop: 256
// columns, or the rows of one round of CTAs, 8 per SM.
constexpr int64_t kMaxLength = INT32_MAX - 4095;
bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxLength; }
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t cdiv(int64_t v, int64_t m) { return (v + m - 1) / m; }

// ------------------------------------------------------------ tensor maps --
// A stack of `z` row-major 16-bit matrices of rows x cols, rows `pitch` and
// matrices `zstride` elements apart.
struct Stack {
  const void* p;
  int64_t rows, cols, pitch, z, zstride;
};

bool make_map(const gemm_ops_s* h, CUtensorMap* m, const Stack& s, bool bf16, uint32_t box_cols,
              uint32_t box_rows, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(s.cols), static_cast<cuuint64_t>(s.rows),
                              static_cast<cuuint64_t>(s.z)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s.pitch) * 2,
                                 static_cast<cuuint64_t>(s.zstride) * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  // Rows whose pitch is not a multiple of 128 bytes straddle L2 lines:
  // promoting their requests to 256 bytes costs more than it saves.
  const CUtensorMapL2promotion l2 = s.pitch % 64 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  auto encode = [&] {
    return reinterpret_cast<EncodeTiledFn>(h->encode)(
        m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
        const_cast<void*>(s.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
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

FusedArgs base_args(const gemm_ops_s* h, const Product& p) {
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
                           const Stack& d, cudaStream_t stream) {
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
  bool ok = make_map(h, &ma, p.a, p.bf16, 64, p.a_mn ? 64 : a_rows) &&
            make_map(h, &mb, p.b, p.bf16, 64, p.b_mn ? 64 : b_rows);
  if (ok && c.p) ok = make_map(h, &mc, c, p.bf16, 64, 32);
  if (ok && d.p)
    ok = Cfg::kSym ? make_map(h, &md, d, p.bf16, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE)
                   : make_map(h, &md, d, p.bf16, 64, 32);
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
  const int64_t fit = Cfg::kCtas == 2 ? h->max_pairs : h->num_sms;
  const int64_t units = Cfg::kSplit > 1 ? items : std::min<int64_t>(items, fit);
  return launch(h, fused_kernel<Cfg>, dim3(static_cast<unsigned>(units * Cfg::kCluster)), dim3(Cfg::kThreads),
                Cfg::kSmemBytes, Cfg::kCluster, stream, ma, mb, mc, md, a);
}

// Which form: the one whose rounds of tiles take the least time by this model,
// in units of 10 ns: a k-block takes a lone CTA 0.27 us (its 32 KB of operands
// through the SM's L2 port), a pair 0.33 us (the tensor pipe), and a tile starts
// and ends in 4 to 7 us.  Of clusters of two CTAs 76 fit at once, of four 36, of
// eight 15.  Lone clusters split a tile only where all fit at once.
//
// The batched products (high and low parts) go by one matrix's tiles alone, so
// that a matrix of a batch gets the same sums as by itself: the number of its
// k-ranges is fixed, and the batch's tiles decide who sums them.
template <int kEpi>
gemm_status_t fused(gemm_ops_s* h, const Product& p, const FusedArgs& a, const Stack& c,
                    const Stack& d, cudaStream_t stream) {
  constexpr bool kBatched = kEpi == kEpiSplit || kEpi == kEpiSplitSym;
  auto tiles = [&](int64_t tm, int64_t tn) { return Pair<kEpi>::kSym ? tn * (tn + 1) / 2 : tm * tn; };
  const int64_t n = kBatched ? 1 : p.batch, kb = cdiv(p.K, 64) * p.segs;
  const int64_t small = tiles(cdiv(p.M, 128), cdiv(p.N, Lone<kEpi>::kOutN)) * n;
  const int64_t big = tiles(cdiv(p.M, 256), cdiv(p.N, Pair<kEpi>::kOutN)) * n;
  const int* most = h->max_split;
  enum { kPairs, kPairs2, kLone, kLone2, kLone4, kLone8, kForms };
  constexpr int64_t kNever = INT64_MAX;
  const int64_t cost[kForms] = {
      h->max_pairs > 0 ? cdiv(big, h->max_pairs) * (33 * kb + 500) : kNever,
      h->max_twos > 0 && kb >= 4 ? cdiv(big, h->max_twos) * (33 * cdiv(kb, 2) + 700) : kNever,
      cdiv(small, h->num_sms) * (27 * kb + 400),
      small <= most[1] && kb >= 4 ? 27 * cdiv(kb, 2) + 550 : kNever,
      small <= most[2] && kb >= (kBatched ? 4 : 8) ? 27 * cdiv(kb, 4) + 550 : kNever,
      !kBatched && small <= std::min(8, most[3]) && kb >= 16 ? 27 * cdiv(kb, 8) + 550 : kNever};
  switch (static_cast<int>(std::min_element(cost, cost + kForms) - cost)) {
    case kPairs: return launch_fused<Pair<kEpi>>(h, p, a, c, d, stream);
    case kPairs2: return launch_fused<TwoPairs<kEpi>>(h, p, a, c, d, stream);
    case kLone2:
      if constexpr (kBatched)
        if (small * p.batch > most[1]) return launch_fused<Lone<kEpi, 1, 2>>(h, p, a, c, d, stream);
      return launch_fused<Lone<kEpi, 2>>(h, p, a, c, d, stream);
    case kLone4:
      if constexpr (kBatched)
        if (small * p.batch > most[2]) return launch_fused<Lone<kEpi, 1, 4>>(h, p, a, c, d, stream);
      return launch_fused<Lone<kEpi, 4>>(h, p, a, c, d, stream);
    case kLone8:
      if constexpr (!kBatched) return launch_fused<Lone<kEpi, 8>>(h, p, a, c, d, stream);
      [[fallthrough]];
    default: return launch_fused<Lone<kEpi>>(h, p, a, c, d, stream);
  }
}

// out = A B^T, rounded to 16 bits.  `early`: operands that may be loaded while
// the previous kernel ends.  A kernel of this file lets the next one start only
// after it has waited for the one before it, so what is complete by then are
// the caller's tensors, and what the last kernel but one wrote.
enum { kEarlyA = 1, kEarlyB = 2 };
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

template <class Cfg>
bool set_attr() {
  return cudaFuncSetAttribute(fused_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg::kSmemBytes) == cudaSuccess;
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

gemm_status_t check_ld(int64_t ld, int64_t cols) {
  if (ld < cols || ld >= (1ll << 30)) return GEMM_ERR_INVALID_ARG;
  return ld % 8 != 0 ? GEMM_ERR_ALIGNMENT : GEMM_OK;
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
