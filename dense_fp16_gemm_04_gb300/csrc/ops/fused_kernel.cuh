// fused_kernel.cuh -- products with fused epilogues on the tensor cores
// (tcgen05) of sm_103a: the matrix work of the gated feed-forward block, of
// its backward pass, of the orthogonalised update and of a vocabulary's loss.
//
//   acc[m, n] = sum over segments s, k of A[m, k; za(s)] B[n, k; zb(s)]
//
// with 16-bit operands (fp16 or bf16) and fp32 sums in tensor memory.  An
// operand is a stack of matrices (third coordinate z), K- or MN-contiguous.
// A segment picks one matrix of each stack, so one launch sums several
// products into the same accumulator.  What becomes of acc is the epilogue:
//
//   kEpiStore    C = alpha acc, rounded to 16 bits.
//   kEpiGlu      acc's columns are gate and up halves of a tile: the gate rows
//                and up rows of w_in are the two matrices of B's stack, and
//                each half of the MMA's N comes from one of them, so a thread
//                of the epilogue finds g and u of the same element in its own
//                TMEM lane.  h = act(g) u, and g, u themselves when kept.
//   kEpiGluBwd   acc = dh; dg = dh u act'(g), du = dh act(g), h = act(g) u from
//                the kept g and u.
//   kEpiSplit    C + c = alpha acc + beta (S + s): C is held as the sum of a
//                high and a low fp16 matrix (22 significant bits), and so is
//                the source S.
//   kEpiSplitSym the same for a symmetric C: only tiles on and above the
//                diagonal are computed, and each is also stored transposed.
//   kEpiLse      acc = logits z: no C, but for each row and each share of a
//                tile's columns their maximum and sum of exponentials, and the
//                row's target logit (xent_kernels.cuh).
//   kEpiXent     acc = logits z: C = a exp(z - lse) - b [column = target].
//   kEpiSum      C = acc or C += acc, fp32.
//   kEpiStoreLive  C = alpha acc with alpha on the device, its rows where row_map
//                says.
// The last three may have fewer rows or k-blocks than the launch was laid out for:
// their number is on the device (live), with the tokens that have a gradient.
//
// What bounds them.  Large products: the tensor cores, and the power they draw
// (gated block of 8192 tokens, 8192 x 16384: 4100 us, 1610 TFLOP/s; its backward
// pass at 4096 x 8192: 2180 us, 1510 TFLOP/s; update of 4096 x 8192, each product
// three: 5100 us, 1410 TFLOP/s).  Few tokens: the weights' bytes (24 tokens,
// 8192 x 16384: 134 us, 6.0 TB/s).  Small ones: a launch's start and end, 4 to 7
// us (update of 512 x 512: 15 dependent products in 115 us).
//
// Few tiles with long K (kSplit = 2, 4 or 8; two pairs: 2): a cluster of kSplit
// CTAs takes one 128 x 128 tile (two pairs one of 256 x 256), each CTA a k-range
// of it, so that more SMs load operands (one SM's loads, 32 KB a k-block against
// 128 clocks of MMAs, bound a lone CTA).  Update of 512 x 512: 115 us; 196 us with
// the k-ranges' partial sums in global memory and a kernel to add them.
// Each CTA then finishes 128 / kSplit of the tile's columns: every CTA sends
// the others their columns of its partial sums through distributed shared
// memory, and after one cluster barrier adds the kSplit partials of its own in
// rank order (the result does not depend on timing) and runs the epilogue on
// them.  In a batch whose tiles fill the device as they are, lone CTAs keep the
// same k-ranges in kParts accumulators side by side and add them in the same
// order: a matrix gets the same sums whatever the batch.
//
// Units (a CTA with a 128-row tile, or a pair of CTAs with a 256-row one) are
// persistent and take tiles round robin.  Inside a CTA: warp 0 loads A and
// warp 2 or 6 loads B (TMA, 128-byte swizzle, a ring of kStages k-blocks), warp 1
// issues tcgen05.mma, warps 4 and on run the epilogue of the tile before (the
// accumulator is double-buffered in TMEM): one or two warps to each quarter of
// its rows, taking its 64-column chunks in turn.  Bounded waits as in
// ../gemm_kernel.cuh: a wait that outlives the timeout records its site and
// every role leaves.
#pragma once

#include "act.cuh"
#include "ptx_ops.cuh"
#include "wait.cuh"

namespace gb300 {
namespace ops {

enum FusedEpi : int {
  kEpiStore = 0,
  kEpiGlu = 1,
  kEpiGluBwd = 2,
  kEpiSplit = 3,
  kEpiSplitSym = 4,
  kEpiLse = 5,
  kEpiXent = 6,
  kEpiSum = 7,
  kEpiStoreLive = 8,
};

constexpr float kLog2e = 1.4426950408889634f;

// What kEpiXent needs of a row: lse log2(e), a, b and the target's column (-1: none).
struct alignas(16) XentRow {
  float lse2, a, b;
  int32_t target;
};

struct FusedArgs {
  int32_t M, N;               // rows and columns of the output (of h for the gated forward)
  int32_t tiles_m, tiles_n;   // tiles of one matrix of the batch
  int32_t per_batch;          // tiles computed per matrix (tiles_m tiles_n, or the triangle)
  int32_t items;              // tiles of the whole batch
  int32_t num_kb;             // 64-deep k-blocks of one segment
  int32_t segs;               // segments (1, or 3: high high + high low + low high)
  // Third coordinate of matrix b of the batch: b a_zb + a_seg[segment] of A's
  // stack, b b_zb + b_seg[segment] of B's, b c_zb (+ 1: low part) of C's.
  int32_t a_zb, b_zb, c_zb;
  int32_t a_seg[3], b_seg[3];
  int32_t group_m;            // raster group height, in tiles
  uint32_t a_tx;              // bytes of A a CTA loads per k-block
  int32_t stages;             // kFlex: k-blocks in flight, A's a_tx bytes apart
  int32_t a_mn, b_mn;         // operand layouts: 0 K-contiguous, 1 MN-contiguous
  // Bit 0, 1, 2: A, B, `live` were complete before the previous kernel of the stream
  // let this one start, and may be loaded before it ends.
  int32_t early;
  int32_t bf16;               // operands and 16-bit outputs are bf16
  int32_t act, save;          // gated epilogues: activation; keep g and u
  float alpha, beta;
  const uint16_t* src;        // kEpiSplit*: S (rows src_ld apart), its low part src_part further,
  int64_t src_ld, src_part;   //   the next matrix of the batch 2 src_part further;
                              // kEpiGluBwd: g and u, [M, 2N]
  // Split clusters store their columns themselves: c the output, or h; d g and
  // u, or dg and du: rows ldd apart, u (du) d_up columns further.
  uint16_t *c, *d;
  int64_t ldd, d_up;
  int64_t ldc, c_z;           // c_z: from one matrix of C's stack to the next
  const float* alpha_p;       // kEpiStoreLive: alpha
  // kLive: rows, or with live_k k (64 of them a block), that the product has (null: all);
  // at least live_min tiles of rows.  row_map: where a row of C goes (null: in place).
  const int32_t *live, *row_map;
  int32_t live_k, live_min;
  int32_t k_slices;           // kEpiSum: the batch is of so many shares of the k-blocks (0: no such batch)
  // kEpiLse: targets [M], their logits [M] and the shares' (maximum, sum) [share][M].
  const int64_t* targets;
  float* target_z;
  float2* shares;
  const XentRow* xent_rows;   // kEpiXent: [M]
  int32_t col_base;           // kEpiXent: column 0 in the vocabulary
  int32_t add;                // kEpiSum: to what is there
  uint32_t* err;
  uint64_t timeout_ns;
  int32_t skip_kb;            // fault injection, -1 = off
};

// A share's running maximum m and sum s of exponentials, s = sum exp(z - m); where
// m is infinite, s = sum exp(z).  Takes in kN more logits.
template <int kN>
__device__ __forceinline__ void lse_take(const float (&z)[kN], float& m, float& s) {
  constexpr int kW = kN < 8 ? kN : 8;
  float tops[kW];
#pragma unroll
  for (int i = 0; i < kW; ++i) tops[i] = z[i];
#pragma unroll
  for (int i = kW; i < kN; ++i) tops[i % kW] = fmaxf(tops[i % kW], z[i]);
  float top = m;  // NaN drops out here, and comes back through s
#pragma unroll
  for (int i = 0; i < kW; ++i) top = fmaxf(top, tops[i]);
  const float ref = isinf(top) ? 0.0f : top;
  const float k = -ref * kLog2e;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kN; ++i) sum[i & 3] += ptx::ex2(fmaf(z[i], kLog2e, k));
  s = fmaf(s, ptx::ex2((m - ref) * kLog2e), (sum[0] + sum[1]) + (sum[2] + sum[3]));
  m = top;
}

// a exp(z - lse), less b at the target: what kEpiXent stores.  A row of no loss and
// no gradient of its lse is zero, whatever its logits.
template <int kN>
__device__ __forceinline__ void xent_columns(const XentRow& r, int32_t col, float (&v)[kN]) {
  const bool none = r.a == 0.0f && r.b == 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float e = r.a * ptx::ex2(fmaf(v[i], kLog2e, -r.lse2));
    v[i] = none ? 0.0f : e;
  }
  const int32_t at = r.target - col;
  if (at >= 0 && at < kN && !none) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i == at) v[i] -= r.b;
  }
}

constexpr int kSumKb = 128;  // 8192 products: 512 steps of the tensor cores
constexpr int kSplitKb = 8;  // 512 products

template <int kCtas_, int kBN_, int kStages_, int kEpi_, int kEpiBufs_, int kSplit_ = 1, int kParts_ = 1>
struct FusedCfg {
  static constexpr int kParts = kParts_;  // accumulators of a tile, one per k-range (0: joined in registers)
  static constexpr int kSplit = kSplit_;  // CTAs sharing a tile, each a k-range
  static constexpr int kCluster = kCtas_ * kSplit_;
  static constexpr int kCtas = kCtas_;
  static constexpr int kBN = kBN_;  // columns of the accumulator
  static constexpr int kStages = kStages_;
  static constexpr int kEpi = kEpi_;
  static constexpr int kEpiBufs = kEpiBufs_;  // 32 x 64 staging buffers per epilogue warp
  static constexpr bool kGlu = kEpi == kEpiGlu;
  static constexpr bool kSym = kEpi == kEpiSplitSym;
  // The loss's products: sums of kPartKb k-blocks at a time, added up in registers.  The
  // tensor cores truncate a sum at each of its K / 16 steps, always towards zero: the loss
  // of one token over 4096 products was off by 9e-6 of itself, of which 16 steps at a time
  // leave 5e-7 (4096 tokens x 4096 x 131072: 2545 -> 2577 us).  The backward pass's logits
  // the same: exp(z - lse) - 1 of a token that the model is sure of is the difference of two
  // numbers that are both off by little.  Of a split cluster, kParts accumulators that are
  // added up as they are sent, up to kSplitKb k-blocks in each; longer ranges (kParts 0)
  // go to registers, kSplitKb at a time (collect_parts).
  //
  // dx and dW: up to kSumKb k-blocks in one accumulator, longer sums in forms of their own
  // (kParts 0; of a split cluster kParts accumulators).  131072 products at a stretch lost 1.5e-4 of dx and 262144
  // 2.6e-4, where fp16 rounds by 2.1e-4; of 8192 at a time 8e-6 are lost.  Every 2048 took
  // longer (16384 tokens x 1024 x 32768 2250 -> 2345 us; at a stretch 2257).  Short
  // sums keep a form without the registers: the 168 of the long one leave no room on an SM
  // for the blocks of the next kernel (128 x 1032 x 8191: 32 us, 41 with the long form).
  static constexpr bool kPartial = kEpi == kEpiLse || kEpi == kEpiXent;
  static constexpr bool kSums = kEpi == kEpiSum || kEpi == kEpiStoreLive;
  static constexpr int kPartKb =
      kPartial ? (kSplit > 1 && kParts == 0 ? kSplitKb : 4) : kSums && kParts != 1 ? kSumKb : 0;
  static constexpr bool kHands = kPartKb > 0 && kParts <= 1;  // partial sums go to registers one by one
  static constexpr bool kCollect = kHands && kSplit > 1;
  static constexpr bool kLive = kEpi == kEpiXent || kEpi == kEpiSum || kEpi == kEpiStoreLive;
  static constexpr bool kReads = kEpi == kEpiGluBwd || kEpi == kEpiSplit || kSym;  // the epilogue reads too
  static constexpr int kOutN = kGlu ? kBN / 2 : kBN;  // output columns per tile
  static constexpr int kBM = 128, kBK = 64;
  static constexpr int kTileM = kBM * kCtas;
  static constexpr int kBRows = kBN / kCtas;
  static constexpr int kABytes = kBM * kBK * 2;
  static constexpr int kBBytes = kBRows * kBK * 2;
  // Eight epilogue warps where few k-blocks make the epilogue the bound (weight
  // gradients of 1000 tokens: -5%); four where K is three times as long and the
  // power cap sets the speed (update of 4096 x 8192: eight cost 2%).
  // Sixteen for 256 columns of logits, of which each thread holds 64 in registers (eight,
  // 128 of them: 4096 x 4096 x 131072 2577 us, 2531 with sixteen).
  static constexpr int kEpiWarps = kEpi == kEpiSplit || kEpi == kEpiSplitSym ? 4 : kPartial && kBN == 256 ? 16 : 8;
  static constexpr int kGroups = kEpiWarps / 4;  // warps per quarter of the rows
  static constexpr int kWarpB = kSplit > 1 ? 6 : 2;  // loads B
  static constexpr int kBufBytes = 32 * 128;
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffEpi = kOffB + kStages * kBBytes;
  static constexpr int kOffBar = kOffEpi + kEpiWarps * kEpiBufs * kBufBytes;
  // Few rows leave room for more k-blocks: their number is the launch's.
  static constexpr bool kFlex =
      kCtas == 1 && (kEpi == kEpiStore || kEpi == kEpiGlu || kEpi == kEpiLse || kEpi == kEpiXent || kEpi == kEpiSum ||
                     kEpi == kEpiStoreLive);
  static constexpr int kMaxStages = !kFlex ? kStages : kEpi == kEpiLse ? 12 : 8;
  static constexpr int kNumBars = 2 * kMaxStages + 5;
  static constexpr int kOffSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kSmemBytes = kOffAbort + 4 + 1024;  // + slack to align the base
  static constexpr int kAccBufs = kParts > 1 ? 1 : 2;  // tiles in tensor memory
  static constexpr int kTmemCols = kAccBufs * (kParts > 0 ? kParts : 1) * kBN;
  // Split clusters end in an epilogue of all eight warps; else warps 4 and on.
  static constexpr int kThreads = kSplit > 1 ? 256 : 128 + 32 * kEpiWarps;
  static constexpr uint32_t kIdesc = ptx::idesc_f16(kTileM, kBN, true);
  static_assert(kSmemBytes <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(kOutN % 64 == 0, "the epilogue works on 64-column chunks");
  static_assert(!kSym || kTileM == kBN, "symmetric tiles are square");
  static_assert(kTmemCols <= 512, "TMEM columns");
  static_assert(kParts == 1 || (kSplit == 1 && (kEpi == kEpiSplit || kEpi == kEpiSplitSym)) ||
                    (kSplit > 1 && kPartKb > 0) || (kSums && kParts == 0),
                "parts");
  // The partials a split CTA receives (a lone one its own among them): 128 rows
  // x 128 columns in all, in the staging buffers' place.
  static_assert(kSplit == 1 || kEpiWarps * kEpiBufs * kBufBytes >= kBM * 128 * 4, "partials");
  static_assert(kSplit == 1 || (kCtas == 1 && kBN == 128) || (kCtas == 2 && kBN == 256 && kSplit == 2),
                "split clusters: lone CTAs on 128 x 128 tiles, two pairs on 256 x 256 ones");
};

// k-blocks of one of the kParts accumulators of a split CTA, of a k-range of n.
template <class Cfg>
__device__ __forceinline__ int32_t part_length(int32_t n) {
  return max(Cfg::kPartKb, (n + Cfg::kParts - 1) / Cfg::kParts);
}

// One tile, and a CTA's k-range of it.
struct FusedItem {
  int32_t mb, nb, batch, kb0, kb1;
};

// What of a launch's size may be on the device.
struct FusedDims {
  int32_t rows, tiles_m, per_batch, items, num_kb;
};

template <class Cfg>
__device__ __forceinline__ FusedDims fused_dims(const FusedArgs& a) {
  FusedDims d = {a.M, a.tiles_m, a.per_batch, a.items, a.num_kb};
  if constexpr (Cfg::kLive) {
    if (a.live) {
      if (!(a.early & 4)) ptx::griddep_wait();
      const int32_t n = *reinterpret_cast<const volatile int32_t*>(a.live);
      if (a.live_k) {
        d.num_kb = max(1, (n + 63) / 64);
      } else {
        d.rows = n;
        d.tiles_m = max(a.live_min, (n + Cfg::kTileM - 1) / Cfg::kTileM);
        d.per_batch = d.tiles_m * a.tiles_n;
        d.items = d.per_batch * max(1, a.k_slices);
      }
    }
  }
  return d;
}

template <class Cfg>
__device__ __forceinline__ FusedItem fused_item(const FusedArgs& a, const FusedDims& d, int32_t t, int32_t rank) {
  FusedItem w;
  const int32_t total = d.num_kb * a.segs;
  w.kb0 = Cfg::kSplit > 1 ? rank * total / Cfg::kSplit : 0;
  w.kb1 = Cfg::kSplit > 1 ? (rank + 1) * total / Cfg::kSplit : total;
  w.batch = t / d.per_batch;
  const int32_t r = t - w.batch * d.per_batch;
  if (Cfg::kEpi == kEpiSum && a.k_slices > 0) {
    w.kb0 = static_cast<int32_t>(static_cast<int64_t>(w.batch) * total / a.k_slices);
    w.kb1 = static_cast<int32_t>(static_cast<int64_t>(w.batch + 1) * total / a.k_slices);
  }
  if constexpr (Cfg::kSym) {
    // Triangle r: column nb holds rows 0 .. nb.
    int32_t j = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
    while ((j + 1) * (j + 2) / 2 <= r) ++j;
    while (j * (j + 1) / 2 > r) --j;
    w.nb = j;
    w.mb = r - j * (j + 1) / 2;
  } else {
    raster(r, d.tiles_m, a.tiles_n, a.group_m, w.mb, w.nb);
  }
  return w;
}

// 2 kN bytes of kN 16-bit values at p (aligned to them).
template <int kN>
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&v)[kN / 2]) {
  if constexpr (kN == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < kN / 8; ++i)
      ptx::st_global_v4(p + 8 * i, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// The epilogue of kN columns of one row, from col0 on: v their sums (gated: of
// the gate, u of the up projection), s0 and s1 what the epilogue reads there.
template <class Cfg, int kN>
__device__ __forceinline__ void finish_columns(const FusedArgs& args, const FusedItem& wi, int32_t row,
                                               int32_t col0, const float (&v)[kN], const float* u,
                                               const uint4* s0, const uint4* s1) {
  const bool bf16 = args.bf16 != 0;
  // Columns come in groups of eight that are in or out together (four, gated
  // over eight CTAs): N is a multiple of 8, or the rows are padded to one.
  constexpr int kG = kN < 8 ? kN : 8;
  if constexpr (Cfg::kEpi == kEpiStore) {
    uint16_t* c = args.c + wi.batch * args.c_zb * args.c_z + static_cast<int64_t>(row) * args.ldc + col0;
#pragma unroll
    for (int i = 0; i < kN; i += kG) {
      uint32_t p[kG / 2];
#pragma unroll
      for (int j = 0; j < kG / 2; ++j)
        p[j] = pack16(bf16, args.alpha * v[i + 2 * j], args.alpha * v[i + 2 * j + 1]);
      if (col0 + i < args.N) store16<kG>(c + i, p);
    }
  } else if constexpr (Cfg::kEpi == kEpiStoreLive) {
    const float alpha = *args.alpha_p;
    uint16_t* c = args.c + static_cast<int64_t>(args.row_map ? args.row_map[row] : row) * args.ldc + col0;
#pragma unroll
    for (int i = 0; i < kN; i += kG) {
      uint32_t p[kG / 2];
#pragma unroll
      for (int j = 0; j < kG / 2; ++j) p[j] = pack16(bf16, alpha * v[i + 2 * j], alpha * v[i + 2 * j + 1]);
      if (col0 + i < args.N) store16<kG>(c + i, p);
    }
  } else if constexpr (Cfg::kEpi == kEpiXent) {
    uint16_t* c = args.c + static_cast<int64_t>(row) * args.ldc + col0;
    float w[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = v[i];
    XentRow r = {};  // behind the last row: zeros, up to a whole k-block of the next product
    if (row < *args.live) r = args.xent_rows[row];
    xent_columns<kN>(r, args.col_base + col0, w);
#pragma unroll
    for (int i = 0; i < kN; i += kG) {
      uint32_t p[kG / 2];
#pragma unroll
      for (int j = 0; j < kG / 2; ++j) p[j] = pack16(bf16, w[i + 2 * j], w[i + 2 * j + 1]);
      if (col0 + i < args.N) store16<kG>(c + i, p);
    }
  } else if constexpr (Cfg::kEpi == kEpiLse) {
    float z[kN], m = -INFINITY, s = 0.0f;
    const int64_t at = args.targets[row] - col0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      z[i] = col0 + i < args.N ? v[i] : -INFINITY;
      if (i == at && col0 + i < args.N) args.target_z[row] = v[i];
    }
    lse_take<kN>(z, m, s);
    args.shares[static_cast<int64_t>(col0 / kN) * args.M + row] = make_float2(m, s);
  } else if constexpr (Cfg::kEpi == kEpiGlu) {
    uint16_t* c = args.c + static_cast<int64_t>(row) * args.ldc + col0;
    uint16_t* d = args.d + static_cast<int64_t>(row) * args.ldd + col0;
#pragma unroll
    for (int i = 0; i < kN; i += kG) {
      uint32_t h[kG / 2], gp[kG / 2], up[kG / 2];
#pragma unroll
      for (int j = 0; j < kG / 2; ++j) {
        const int k = i + 2 * j;
        h[j] = pack16(bf16, act_value(args.act, v[k]) * u[k], act_value(args.act, v[k + 1]) * u[k + 1]);
        gp[j] = pack16(bf16, v[k], v[k + 1]);
        up[j] = pack16(bf16, u[k], u[k + 1]);
      }
      if (col0 + i < args.N) {
        store16<kG>(c + i, h);
        if (args.save) {
          store16<kG>(d + i, gp);
          store16<kG>(d + args.d_up + i, up);
        }
      }
    }
  } else if constexpr (Cfg::kEpi == kEpiGluBwd) {
    uint16_t* c = args.c + static_cast<int64_t>(row) * args.ldc + col0;
    uint16_t* d = args.d + static_cast<int64_t>(row) * args.ldd + col0;
#pragma unroll
    for (int i = 0; i < kN; i += kG) {
      if (col0 + i >= args.N) break;
      const uint4 gv = s0[i / 8], uv = s1[i / 8];
      const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, uw[4] = {uv.x, uv.y, uv.z, uv.w};
      uint32_t h[kG / 2], dg[kG / 2], du[kG / 2];
#pragma unroll
      for (int j = 0; j < kG / 2; ++j) {
        const float2 gf = unpack16(bf16, gw[j]), uf = unpack16(bf16, uw[j]);
        float a0, a1, s0, s1;
        act_both(args.act, gf.x, a0, s0);
        act_both(args.act, gf.y, a1, s1);
        const float d0 = v[i + 2 * j], d1 = v[i + 2 * j + 1];
        dg[j] = pack16(bf16, d0 * uf.x * s0, d1 * uf.y * s1);
        du[j] = pack16(bf16, d0 * a0, d1 * a1);
        h[j] = pack16(bf16, a0 * uf.x, a1 * uf.y);
      }
      store16<kG>(c + i, h);
      store16<kG>(d + i, dg);
      store16<kG>(d + args.d_up + i, du);
    }
  } else {
    static_assert(Cfg::kEpi == kEpiSplit || Cfg::kEpi == kEpiSplitSym, "no other epilogue splits a tile");
    uint16_t* base = args.c + wi.batch * args.c_zb * args.c_z;
    uint16_t* c = base + static_cast<int64_t>(row) * args.ldc + col0;
#pragma unroll
    for (int i = 0; i < kN; i += kG) {
      if (col0 + i >= args.N) break;
      float x[kG];
#pragma unroll
      for (int j = 0; j < kG; ++j) x[j] = args.alpha * v[i + j];
      if (args.beta != 0.0f) {
        const uint4 a = s0[i / 8], b = s1[i / 8];
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < kG / 2; ++j) {
          const float2 hf = unpack16(false, aw[j]), lf = unpack16(false, bw[j]);
          x[2 * j] = fmaf(args.beta, hf.x + lf.x, x[2 * j]);
          x[2 * j + 1] = fmaf(args.beta, hf.y + lf.y, x[2 * j + 1]);
        }
      }
      uint32_t hi[kG / 2], lo[kG / 2];
#pragma unroll
      for (int j = 0; j < kG / 2; ++j) {
        hi[j] = pack16(false, x[2 * j], x[2 * j + 1]);
        const float2 back = unpack16(false, hi[j]);
        lo[j] = pack16(false, x[2 * j] - back.x, x[2 * j + 1] - back.y);
      }
      store16<kG>(c + i, hi);
      store16<kG>(c + args.c_z + i, lo);
      if constexpr (Cfg::kSym) {
        // Transposed: a warp's 32 rows are 64 contiguous bytes of each column.
        if (wi.mb != wi.nb) {
#pragma unroll
          for (int j = 0; j < kG; ++j) {
            uint16_t* t = base + static_cast<int64_t>(col0 + i + j) * args.ldc + row;
            if (col0 + i + j < args.N) {
              ptx::st_global_b16(t, static_cast<uint16_t>(hi[j / 2] >> (16 * (j & 1))));
              ptx::st_global_b16(t + args.c_z, static_cast<uint16_t>(lo[j / 2] >> (16 * (j & 1))));
            }
          }
        }
      }
    }
  }
}

// What the epilogue of kN columns reads: S and its low part, or g and u.
template <class Cfg, int kN>
__device__ __forceinline__ void read_columns(const FusedArgs& args, const FusedItem& wi, int32_t row,
                                             int32_t col0, uint4* s0, uint4* s1) {
  if constexpr (Cfg::kReads) {
    const bool gated = Cfg::kEpi == kEpiGluBwd;
    const int64_t second = gated ? args.N : args.src_part;
    const uint16_t* src = args.src + (gated ? 0 : static_cast<int64_t>(wi.batch) * 2 * args.src_part) +
                          static_cast<int64_t>(row) * args.src_ld + col0;
    if (gated || args.beta != 0.0f) {
#pragma unroll
      for (int i = 0; i < kN / 8; ++i)
        if (col0 + 8 * i < args.N) {
          s0[i] = ptx::ld_global_v4_u32(src + 8 * i);
          s1[i] = ptx::ld_global_v4_u32(src + second + 8 * i);
        }
    }
  }
}

// 16 columns of a split CTA's sums: its partial ones added up in order.
template <class Cfg>
__device__ __forceinline__ void load_parts(const FusedItem& wi, uint32_t t, uint32_t (&v)[16]) {
  ptx::tmem_ld_32x32b_x16(t, v);
  ptx::tmem_wait_ld(v);
  if constexpr (Cfg::kParts > 1) {
    const int32_t n = wi.kb1 - wi.kb0, length = part_length<Cfg>(n);
    for (int32_t q = 1; q * length < n; ++q) {
      uint32_t u[16];
      ptx::tmem_ld_32x32b_x16(t + q * Cfg::kBN, u);
      ptx::tmem_wait_ld(u);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
    }
  }
}

// A split CTA's partial sums of logits: four warps (2 to 5) add them up while the next are
// made, each 32 rows of 128 columns, and send them as split_epilogue would.  The loss of
// one token, 16384 x 9000, is off by 3e-6 so; with four accumulators for the whole range it
// was by 1.3e-5 (52.0 -> 52.7 us; 3 tokens, 8192 x 5000: 21.4 -> 22.2).
template <class Cfg>
__device__ __forceinline__ void collect_parts(const FusedItem& wi, int32_t rank, uint32_t tmem_base, uint32_t recv,
                                              uint32_t tfull0, uint32_t tempty0, const Watch& w) {
  constexpr int kCols = 128 / Cfg::kSplit;
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  float z[128];
#pragma unroll
  for (int i = 0; i < 128; ++i) z[i] = 0.0f;
  int32_t acc_iter = 0;
  for (int32_t kb = wi.kb0; kb < wi.kb1; kb += Cfg::kPartKb, ++acc_iter) {
    const int buf = acc_iter % Cfg::kAccBufs;
    const uint32_t use_par = static_cast<uint32_t>((acc_iter / Cfg::kAccBufs) & 1);
    if (!wait_bar_warp<false>(tfull0 + 8u * buf, use_par, w, kSiteTmemFull, wi.mb)) return;
    ptx::tc_fence_after();
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * Cfg::kBN);
#pragma unroll
    for (int c = 0; c < 128; c += 16) {
      uint32_t v[16];
      ptx::tmem_ld_32x32b_x16(t_row + c, v);
      ptx::tmem_wait_ld(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) z[c + i] += __uint_as_float(v[i]);
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(tempty0 + 8u * buf);
  }
  const uint32_t mine = recv + static_cast<uint32_t>(rank * (kCols / 4) * 128 + q * 32 + lane) * 16u;
#pragma unroll
  for (int c = 0; c < 128; c += 4)
    ptx::st_shared_cluster_v4(ptx::mapa(mine + static_cast<uint32_t>(c % kCols / 4 * 128) * 16u, static_cast<uint32_t>(c / kCols)),
                              __float_as_uint(z[c]), __float_as_uint(z[c + 1]), __float_as_uint(z[c + 2]),
                              __float_as_uint(z[c + 3]));
}

// The end of a split cluster's tile, run by all 256 threads of each CTA: lone
// CTAs.
template <class Cfg>
__device__ __forceinline__ void split_epilogue(const FusedArgs& args, const FusedDims& dims, int32_t unit, int32_t rank,
                                               uint32_t tmem_base, uint32_t recv, uint32_t tfull,
                                               const Watch& w) {
  constexpr int kS = Cfg::kSplit;
  constexpr int kCols = Cfg::kBN / kS;  // accumulator columns this CTA finishes
  constexpr int kHalfCols = kCols / 2;  // gated: gate columns, then as many up columns
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::griddep_wait();  // reads S, g and u; writes the outputs
  ptx::griddep_launch_dependents();
  const FusedItem wi = fused_item<Cfg>(args, dims, unit, rank);
  const bool ok = Cfg::kCollect || wait_bar_warp<false>(tfull, 0u, w, kSiteTmemFull, unit);
  if (ok && !Cfg::kCollect) {
    // Send: warp quarter q owns 32 rows, warps 0-3 columns 0-63, warps 4-7 the
    // rest (gated: gate, up).  Receiver's slot: [source][4 columns][row][16 B],
    // so a warp writes 512 contiguous bytes at a time.
    ptx::tc_fence_after();
    const int q = warp & 3, side = warp >> 2;
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + side * 64;
    const uint32_t mine = recv + static_cast<uint32_t>(rank * (kCols / 4) * 128 + q * 32 + lane) * 16u;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t v[16];
      load_parts<Cfg>(wi, t_row + g * 16, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = g * 16 + j * 4;  // of this side's 64
        int to, at;                    // receiving CTA, its 4-column group
        if (Cfg::kGlu) {
          to = c / kHalfCols;
          at = (c % kHalfCols) / 4 + side * (kHalfCols / 4);
        } else {
          to = (side * 64 + c) / kCols;
          at = (side * 64 + c) % kCols / 4;
        }
        ptx::st_shared_cluster_v4(ptx::mapa(mine + static_cast<uint32_t>(at * 128) * 16u, static_cast<uint32_t>(to)),
                                  v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
  }
  // Thread (row, half) finishes half of the CTA's columns.  What the epilogue
  // reads comes in while the partials do.
  constexpr int kN = Cfg::kGlu ? kHalfCols / 2 : kCols / 2;
  const int r = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int32_t row = wi.mb * Cfg::kBM + r;
  const int32_t col0 = wi.nb * Cfg::kOutN + rank * (Cfg::kOutN / kS) + half * kN;
  const bool in = row < (Cfg::kEpi == kEpiXent ? args.M : dims.rows) && (col0 < args.N || Cfg::kEpi == kEpiLse);  // (every share is written)
  uint4 s0[Cfg::kReads ? kN / 8 : 1], s1[Cfg::kReads ? kN / 8 : 1];
  if (in) read_columns<Cfg, kN>(args, wi, row, col0, s0, s1);
  ptx::cluster_sync();
  if (!ok || !in || (Cfg::kCollect && *w.abort)) return;
  auto sum = [&](int first4, float (&v)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = 0.0f;
#pragma unroll
    for (int s = 0; s < kS; ++s)
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float4 p = ptx::ld_shared_v4_f32(
            recv + static_cast<uint32_t>((s * (kCols / 4) + first4 + i) * 128 + r) * 16u);
        v[4 * i] += p.x, v[4 * i + 1] += p.y, v[4 * i + 2] += p.z, v[4 * i + 3] += p.w;
      }
  };
  float v[kN], u[Cfg::kGlu ? kN : 1];
  sum(half * (kN / 4), v);
  if constexpr (Cfg::kGlu) sum(kHalfCols / 4 + half * (kN / 4), u);
  finish_columns<Cfg, kN>(args, wi, row, col0, v, u, s0, s1);
}

// The same for two pairs of CTAs, each with half of the k-blocks of a 256 x 256
// tile: pair k finishes half k of its columns (gated: of the gate's and of the
// up projection's), and each CTA sends its 128 rows of the other half to the
// CTA of the same rows in the other pair.  A sum of two: its order is free.
template <class Cfg>
__device__ __forceinline__ void pair_split_epilogue(const FusedArgs& args, const FusedDims& dims, int32_t unit, int32_t k, uint32_t cta,
                                                    uint32_t tmem_base, uint32_t recv, uint32_t tfull,
                                                    const Watch& w) {
  constexpr int kOut = Cfg::kOutN / 2;           // output columns a pair finishes
  constexpr int kN = kOut / 2;                   // and a thread
  constexpr int kSide = Cfg::kGlu ? 128 : 64;    // accumulator columns between the two sides' first
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, side = warp >> 2;
  const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const FusedItem wi = fused_item<Cfg>(args, dims, unit, k);
  const bool ok = wait_bar_warp<true>(tfull, 0u, w, kSiteTmemFull, unit);
  const int r = q * 32 + lane;
  if (ok) {
    // Sides: 64 columns each (gated: gate and up).  Slot: [4 columns][row][16 B].
    ptx::tc_fence_after();
    const uint32_t to = ptx::mapa(recv, static_cast<uint32_t>((k ^ 1) * 2) + cta) +
                        static_cast<uint32_t>(side * 16 * 128 + r) * 16u;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t v[16];
      load_parts<Cfg>(wi, t_row + (k ^ 1) * kOut + side * kSide + g * 16, v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ptx::st_shared_cluster_v4(to + static_cast<uint32_t>((g * 4 + j) * 128) * 16u, v[4 * j], v[4 * j + 1],
                                  v[4 * j + 2], v[4 * j + 3]);
    }
  }
  const int32_t row = wi.mb * Cfg::kTileM + static_cast<int32_t>(cta) * Cfg::kBM + r;
  const int32_t col0 = wi.nb * Cfg::kOutN + k * kOut + side * kN;
  const bool in = row < dims.rows && col0 < args.N;
  uint4 s0[Cfg::kReads ? kN / 8 : 1], s1[Cfg::kReads ? kN / 8 : 1];
  if (in) read_columns<Cfg, kN>(args, wi, row, col0, s0, s1);
  ptx::cluster_sync();
  if (!ok) return;
  auto sum = [&](int col, int group4, float (&v)[16]) {  // every lane: tensor memory
    uint32_t t[16];
    load_parts<Cfg>(wi, t_row + col, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 p = ptx::ld_shared_v4_f32(recv + static_cast<uint32_t>((group4 + i) * 128 + r) * 16u);
      v[4 * i] = __uint_as_float(t[4 * i]) + p.x;
      v[4 * i + 1] = __uint_as_float(t[4 * i + 1]) + p.y;
      v[4 * i + 2] = __uint_as_float(t[4 * i + 2]) + p.z;
      v[4 * i + 3] = __uint_as_float(t[4 * i + 3]) + p.w;
    }
  };
#pragma unroll
  for (int c = 0; c < kN; c += 16) {
    float v[16], u[16];
    sum(k * kOut + side * kN + c, (side * kN + c) / 4, v);
    if constexpr (Cfg::kGlu) sum(128 + k * kOut + side * kN + c, 16 + (side * kN + c) / 4, u);
    if (in)
      finish_columns<Cfg, 16>(args, wi, row, col0 + c, v, u, s0 + (Cfg::kReads ? c / 8 : 0),
                              s1 + (Cfg::kReads ? c / 8 : 0));
    __syncwarp();
  }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    fused_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD,
                 const FusedArgs args) {
  const int S = Cfg::kFlex ? args.stages : Cfg::kStages;
  const uint32_t a_stage = Cfg::kFlex ? args.a_tx : Cfg::kABytes;
  const uint32_t off_b = Cfg::kFlex ? S * a_stage : Cfg::kOffB;
  constexpr int kBars = Cfg::kMaxStages;
  constexpr bool kPair = Cfg::kCtas == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr bool kCluster = Cfg::kCluster > 1;
  const uint32_t crank = kCluster ? ptx::cluster_ctarank() : 0u;
  const uint32_t cta = kPair ? crank & 1u : 0u;  // 0: issues the MMAs
  const uint32_t leader = kPair ? crank & ~1u : 0u;  // the pair's CTA that does
  const uint16_t pair_mask = static_cast<uint16_t>(0x3u << leader);
  const int32_t rank = Cfg::kSplit > 1 ? static_cast<int32_t>(crank) / Cfg::kCtas : 0;  // k-range
  const int32_t unit = kCluster ? static_cast<int32_t>(ptx::cluster_id_x()) : static_cast<int32_t>(blockIdx.x);
  const int32_t units = kCluster ? static_cast<int32_t>(ptx::num_clusters_x()) : static_cast<int32_t>(gridDim.x);

  const uint32_t bar0 = sb + Cfg::kOffBar;
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kBars + s); };
  auto bar_tfull = [&](int b) { return bar0 + 8u * (2 * kBars + b); };
  auto bar_tempty = [&](int b) { return bar0 + 8u * (2 * kBars + 2 + b); };
  const uint32_t bar_mma_done = bar0 + 8u * (2 * kBars + 4);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffAbort);
  const Watch w{abort_flag, args.err, args.timeout_ns};

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmC);
    ptx::prefetch_tmap(&tmD);
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(bar_full(s), 2);  // the A and B producers of the leader
      ptx::mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar_tfull(b), 1);
      ptx::mbar_init(bar_tempty(b), Cfg::kCollect ? 4 : Cfg::kEpiWarps * Cfg::kCtas);
    }
    ptx::mbar_init(bar_mma_done, 1);
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc<Cfg::kCtas>(sb + Cfg::kOffSlot, Cfg::kTmemCols);
    ptx::tmem_relinquish<Cfg::kCtas>();
  }
  ptx::tc_fence_before();
  if constexpr (kCluster)
    ptx::cluster_sync();  // every CTA runs, its barriers set up, before another uses its memory
  else
    __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffSlot);
  const FusedDims dims = fused_dims<Cfg>(args);

  if (warp == 0 || warp == Cfg::kWarpB) {
    // ------------------------------------------------------- TMA producers --
    const bool is_a = warp == 0;
    const CUtensorMap* tm = is_a ? &tmA : &tmB;
    const bool mn = is_a ? args.a_mn != 0 : args.b_mn != 0;
    const uint32_t op_bytes = is_a ? a_stage : Cfg::kBBytes;
    const uint32_t op_base = sb + (is_a ? Cfg::kOffA : off_b);
    const uint32_t op_tx = (is_a ? args.a_tx : op_bytes) * Cfg::kCtas;
    // The operand's rows arrive as kBoxes boxes per stage.  Gated forward, B:
    // the gate rows and up rows of the same columns of h (a pair's CTAs load
    // one half each, a lone CTA both); then the row and the matrix differ.
    constexpr int kGluBoxes = kPair ? 1 : 2;
    if (!(args.early & (is_a ? 1 : 2))) {
      ptx::griddep_wait();
      ptx::griddep_launch_dependents();
    }
    int stage = 0;
    uint32_t phase = 0;
    int64_t fills = 0;
    bool ok = true, first_item = true;
    for (int32_t it = unit; ok && it < dims.items; it += units) {
      const FusedItem wi = fused_item<Cfg>(args, dims, it, rank);
      int32_t row;
      const int32_t z0 = wi.batch * (is_a ? args.a_zb : args.b_zb);
      if (is_a)
        row = wi.mb * Cfg::kTileM + static_cast<int32_t>(cta) * Cfg::kBM;
      else if (Cfg::kGlu)
        row = wi.nb * Cfg::kOutN;
      else
        row = wi.nb * Cfg::kBN + static_cast<int32_t>(cta) * Cfg::kBRows;
      int32_t seg = wi.kb0 / dims.num_kb, k = wi.kb0 - seg * dims.num_kb;
      for (int32_t kb = wi.kb0; kb < wi.kb1; ++kb) {
        if (!wait_bar_warp<kPair>(bar_empty(stage), phase ^ 1u, w, kSiteEmpty, it)) {
          ok = false;
          break;
        }
        const bool skip = args.skip_kb == kb && first_item && unit == 0 && cta == 0;
        if (!skip && ptx::elect_one()) {
          const uint32_t dst = op_base + static_cast<uint32_t>(stage) * op_bytes;
          const int32_t z = z0 + (is_a ? args.a_seg[seg] : args.b_seg[seg]);
          uint32_t full = bar_full(stage);
          if constexpr (kPair) {
            full = ptx::mapa(full, leader);
            if (cta == 0) ptx::mbar_arrive_expect_tx(bar_full(stage), op_tx);
          } else {
            ptx::mbar_arrive_expect_tx(full, op_tx);
          }
          auto load = [&](uint32_t d, int32_t c0, int32_t c1, int32_t c2) {
            if constexpr (kPair)
              ptx::tma_load_3d_pair(d, tm, full, c0, c1, c2);
            else
              ptx::tma_load_3d(d, tm, full, c0, c1, c2);
          };
          if (Cfg::kGlu && !is_a) {
#pragma unroll
            for (int b = 0; b < kGluBoxes; ++b)
              load(dst + b * (Cfg::kBBytes / kGluBoxes), k * Cfg::kBK, row,
                   static_cast<int32_t>(cta) + b);
          } else if (mn) {
            // MN-contiguous: 64 x 64 boxes, 8 KB apart.
            const int boxes = (is_a ? Cfg::kBM : Cfg::kBRows) / 64;
            for (int g = 0; g < boxes; ++g) load(dst + g * 8192, row + 64 * g, k * Cfg::kBK, z);
          } else {
            load(dst, k * Cfg::kBK, row, z);
          }
        }
        __syncwarp();
        if (++k == dims.num_kb) {
          k = 0;
          ++seg;
        }
        ++fills;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      first_item = false;
    }
    // Drain: the MMAs have released the last fills, or (aborting) the loads
    // have landed.
    const int64_t n = fills < S ? fills : S;
    for (int64_t f = fills - n; f < fills; ++f) {
      const int s = static_cast<int>(f % S);
      const uint32_t par = static_cast<uint32_t>((f / S) & 1);
      if (ok) ok = wait_bar_warp<kPair>(bar_empty(s), par, w, kSiteDrain, -1);
      if (!ok && cta == 0)
        wait_bar_warp<kPair>(bar_full(s), par, w, kSiteDrain, -1, /*honor_abort=*/false);
    }
  } else if (warp == 1) {
    if (cta == 0) {
      // ------------------------------------------------------- MMA issuer --
      const uint32_t idesc = Cfg::kIdesc | (args.a_mn ? ptx::kIdescAMnMajor : 0u) |
                             (args.b_mn ? ptx::kIdescBMnMajor : 0u) |
                             (args.bf16 ? ptx::kIdescBf16 : 0u);
      const uint64_t a_kstep = args.a_mn ? 128u : 2u;
      const uint64_t b_kstep = args.b_mn ? 128u : 2u;
      const uint64_t a_desc0 = args.a_mn ? ptx::sw128_mnmajor_desc(sb + Cfg::kOffA)
                                         : ptx::sw128_kmajor_desc(sb + Cfg::kOffA);
      const uint64_t b_desc0 = args.b_mn ? ptx::sw128_mnmajor_desc(sb + off_b)
                                         : ptx::sw128_kmajor_desc(sb + off_b);
      const uint64_t a_desc_stage = a_stage >> 4;
      constexpr uint64_t kBDescStage = Cfg::kBBytes >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int32_t acc_iter = 0;
      bool ok = true;
      for (int32_t it = unit; ok && it < dims.items; it += units) {
        const FusedItem wi = fused_item<Cfg>(args, dims, it, rank);
        int32_t kb = wi.kb0;
        do {  // once, or for each partial sum
          const int32_t end = Cfg::kHands ? min(wi.kb1, kb + Cfg::kPartKb) : wi.kb1;
          const int buf = acc_iter % Cfg::kAccBufs;
          const uint32_t use_par = static_cast<uint32_t>((acc_iter / Cfg::kAccBufs) & 1);
          if (!wait_bar_warp<kPair>(bar_tempty(buf), use_par ^ 1u, w, kSiteTmemEmpty, it)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * Cfg::kBN);
          int32_t first = kb, part = 0;  // first k-block of the current accumulator
          for (; kb < end; ++kb) {
            if (Cfg::kParts > 1 && kb == (Cfg::kPartKb > 0 ? first + part_length<Cfg>(wi.kb1 - wi.kb0)
                                                           : (part + 1) * wi.kb1 / Cfg::kParts)) {
              ++part;
              first = kb;
              d_tmem += Cfg::kBN;
            }
            if (!wait_bar_warp<kPair>(bar_full(stage), phase, w, kSiteFull, it)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint64_t a_desc = a_desc0 + a_desc_stage * static_cast<uint32_t>(stage);
            const uint64_t b_desc = b_desc0 + kBDescStage * static_cast<uint32_t>(stage);
            const uint32_t acc_first = kb != first ? 1u : 0u;
            if (ptx::elect_one()) {
#pragma unroll
              for (int k = 0; k < Cfg::kBK / 16; ++k)
                ptx::mma_f16<Cfg::kCtas>(d_tmem, a_desc + a_kstep * k, b_desc + b_kstep * k, idesc,
                                         k != 0 ? 1u : acc_first);
              if constexpr (kPair)
                ptx::mma_commit_pair(bar_empty(stage), pair_mask);
              else
                ptx::mma_commit(bar_empty(stage));
            }
            __syncwarp();
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (ptx::elect_one()) {
            if constexpr (kPair)
              ptx::mma_commit_pair(bar_tfull(buf), pair_mask);
            else
              ptx::mma_commit(bar_tfull(buf));
          }
          __syncwarp();
          ++acc_iter;
        } while (kb < wi.kb1);
      }
      // Every MMA has finished before tensor memory is freed.
      if (ptx::elect_one()) {
        if constexpr (kPair)
          ptx::mma_commit_pair(bar_mma_done, static_cast<uint16_t>(1u << leader));
        else
          ptx::mma_commit(bar_mma_done);
      }
      __syncwarp();
      wait_bar_warp<kPair>(bar_mma_done, 0u, w, kSiteMmaDone, -1, /*honor_abort=*/false);
    }
  } else if (Cfg::kCollect && warp >= 2 && warp < 6) {
    if constexpr (Cfg::kCollect)
      if (unit < dims.items)
        collect_parts<Cfg>(fused_item<Cfg>(args, dims, unit, rank), rank, tmem_base, sb + Cfg::kOffEpi, bar_tfull(0),
                           bar_tempty(0), w);
  } else if (Cfg::kSplit == 1 && warp >= 4) {
    // ------------------------------------------------------------ epilogue --
    ptx::griddep_wait();  // reads S, g and u; writes the outputs
    ptx::griddep_launch_dependents();
    const int q = warp & 3;  // this warp may touch TMEM lanes 32q .. 32q+31 only
    const int group = (warp - 4) >> 2;  // which of the two warps of quarter q
    const uint32_t stage_base =
        sb + Cfg::kOffEpi + static_cast<uint32_t>((warp - 4) * Cfg::kEpiBufs * Cfg::kBufBytes);
    const uint32_t tempty_bar0 = kPair ? ptx::mapa(bar_tempty(0), leader) : bar_tempty(0);
    const bool bf16 = args.bf16 != 0;
    const float alpha = Cfg::kEpi == kEpiStoreLive ? *args.alpha_p : args.alpha;
    uint32_t next_buf = 0, used = 0;
    int32_t acc_iter = 0;
    // The next free staging buffer: once the store that last read it is done.
    auto take_buf = [&]() {
      if (used >= Cfg::kEpiBufs && lane == 0) ptx::bulk_wait_group_read<Cfg::kEpiBufs - 1>();
      __syncwarp();
      const uint32_t b = stage_base + next_buf * Cfg::kBufBytes;
      next_buf = next_buf + 1 == Cfg::kEpiBufs ? 0 : next_buf + 1;
      ++used;
      return b;
    };
    // A 32 x 64 chunk (row `lane`, columns in pairs: word(0) .. word(31)) through a
    // swizzled buffer to rows row0.., columns col0.. of matrix z.  Every buffer taken
    // commits one group, empty where nothing of the chunk is in range, so that
    // the count in take_buf holds.
    auto store_words = [&](const CUtensorMap* m, auto word, int32_t col0, int32_t row0, int32_t z, bool in) {
      const uint32_t sbuf = take_buf();
      const uint32_t row_addr = sbuf + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        ptx::st_shared_v4(row_addr + ((static_cast<uint32_t>(j) ^ (lane & 7u)) << 4), word(4 * j), word(4 * j + 1),
                          word(4 * j + 2), word(4 * j + 3));
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (in) {
          if (Cfg::kEpi == kEpiSum && args.add)
            ptx::tma_add_3d(m, sbuf, col0, row0, z);
          else
            ptx::tma_store_3d(m, sbuf, col0, row0, z);
        }
        ptx::bulk_commit_group();
      }
    };
    auto store_chunk = [&](const CUtensorMap* m, const uint32_t (&packed)[32], int32_t col0, int32_t row0, int32_t z,
                           bool in) { store_words(m, [&](int i) { return packed[i]; }, col0, row0, z, in); };
    // The same chunk transposed: 64 rows of 32 columns, unswizzled (a warp's
    // 2-byte stores of one column are 64 contiguous bytes).
    auto store_chunk_t = [&](const uint32_t (&packed)[32], int32_t col0, int32_t row0, int32_t z,
                             bool in) {
      const uint32_t sbuf = take_buf();
      const uint32_t at = sbuf + static_cast<uint32_t>(lane) * 2u;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        ptx::st_shared_u16(at + (2 * j) * 64u, static_cast<uint16_t>(packed[j]));
        ptx::st_shared_u16(at + (2 * j + 1) * 64u, static_cast<uint16_t>(packed[j] >> 16));
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (in) ptx::tma_store_3d(&tmD, sbuf, row0, col0, z);
        ptx::bulk_commit_group();
      }
    };
    // dx, dW: a 32 x 64 chunk of sums.
    auto store_sums = [&](auto sum, int32_t col0, int32_t row0, int32_t row, bool row_in, int32_t batch) {
      if constexpr (Cfg::kEpi == kEpiSum) {
#pragma unroll
        for (int half = 0; half < 64; half += 32)
          store_words(&tmC, [&](int i) { return __float_as_uint(sum(half + i)); }, col0 + half, row0, batch * args.c_zb,
                      col0 + half < args.N);
      } else if constexpr (Cfg::kEpi == kEpiStoreLive) {
        auto word = [&](int i) { return pack16(bf16, alpha * sum(2 * i), alpha * sum(2 * i + 1)); };
        if (!args.row_map) {
          store_words(&tmC, word, col0, row0, 0, true);
        } else if (row_in) {  // each row to its own place: 128 bytes a lane
          uint16_t* to = args.c + static_cast<int64_t>(args.row_map[row]) * args.ldc + col0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col0 + 8 * j < args.N)  // (a multiple of 8)
              ptx::st_global_v4(to + 8 * j, word(4 * j), word(4 * j + 1), word(4 * j + 2), word(4 * j + 3));
        }
      }
    };
    if constexpr (Cfg::kHands) {
      // Each warp for itself: 32 rows, and this group's columns of the tile.
      constexpr int kCols = Cfg::kOutN / Cfg::kGroups;
      constexpr int kLoad = kCols > 64 ? 8 : 16;  // (128 sums and 16 loads do not fit in registers)
      bool ok = true;
      for (int32_t it = unit; ok && it < dims.items; it += units) {
        const FusedItem wi = fused_item<Cfg>(args, dims, it, rank);
        const int32_t row0 = wi.mb * Cfg::kTileM + static_cast<int32_t>(cta) * Cfg::kBM + q * 32, row = row0 + lane;
        const int32_t col0 = wi.nb * Cfg::kOutN + group * kCols;
        const bool row_in = row < dims.rows;
        const bool idle = row0 >= dims.rows || col0 >= args.N;  // none of the warp's sums counts
        int64_t target = -1;
        XentRow xr = {};
        if (row_in) {
          if constexpr (Cfg::kEpi == kEpiLse) target = args.targets[row] - col0;
          if constexpr (Cfg::kEpi == kEpiXent) xr = args.xent_rows[row];
        }
        float z[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) z[i] = 0.0f;
        for (int32_t kb = wi.kb0; kb < wi.kb1; kb += Cfg::kPartKb) {
          const int buf = acc_iter % Cfg::kAccBufs;
          const uint32_t use_par = static_cast<uint32_t>((acc_iter / Cfg::kAccBufs) & 1);
          ++acc_iter;
          ok = wait_bar_warp<kPair>(bar_tfull(buf), use_par, w, kSiteTmemFull, it);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                 static_cast<uint32_t>(buf * Cfg::kBN + group * kCols);
          if (!idle) {
#pragma unroll
            for (int c = 0; c < kCols; c += kLoad) {
              uint32_t v[kLoad];
              if constexpr (kLoad == 8)
                ptx::tmem_ld_32x32b_x8(t_row + c, v);
              else
                ptx::tmem_ld_32x32b_x16(t_row + c, v);
              ptx::tmem_wait_ld(v);
#pragma unroll
              for (int i = 0; i < kLoad; ++i) z[c + i] += __uint_as_float(v[i]);
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair)
              ptx::mbar_arrive_cluster(tempty_bar0 + 8u * buf);
            else
              ptx::mbar_arrive(tempty_bar0 + 8u * buf);
          }
        }
        if (!ok) break;
        if constexpr (Cfg::kEpi == kEpiLse) {
          // No lane's target is among these columns but for a few tiles of a row.
          const bool here = target >= 0 && target < kCols && target < args.N - col0;
          if (__any_sync(0xffffffffu, here)) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (here && target == i) args.target_z[row] = z[i];
          }
          if (col0 + kCols > args.N) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) z[i] = col0 + i < args.N ? z[i] : -INFINITY;
          }
          float share_m = -INFINITY, share_s = 0.0f;
          if (!idle) lse_take<kCols>(z, share_m, share_s);
          if (row_in)
            args.shares[(static_cast<int64_t>(wi.nb) * Cfg::kGroups + group) * args.M + row] =
                make_float2(share_m, share_s);
        } else if constexpr (Cfg::kSums) {
#pragma unroll
          for (int c = 0; c < kCols; c += 64)
            if (!idle && col0 + c < args.N)
              store_sums([&](int i) { return z[c + i]; }, col0 + c, row0, row, row_in, wi.batch);
        } else if (row0 < args.M && col0 < args.N) {
          // Rows behind the last: zeros, up to a whole k-block of the next product.
          static_assert(Cfg::kEpi != kEpiXent || kCols == 64, "one staging buffer");
          const uint32_t sbuf = take_buf();
          xent_columns<kCols>(xr, args.col_base + col0, z);
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j) {
            const uint32_t at = sbuf + static_cast<uint32_t>(lane) * 128u + ((static_cast<uint32_t>(j) ^ (lane & 7u)) << 4);
            ptx::st_shared_v4(at, pack16(bf16, z[8 * j], z[8 * j + 1]), pack16(bf16, z[8 * j + 2], z[8 * j + 3]),
                              pack16(bf16, z[8 * j + 4], z[8 * j + 5]), pack16(bf16, z[8 * j + 6], z[8 * j + 7]));
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_3d(&tmC, sbuf, col0, row0, 0);
            ptx::bulk_commit_group();
          }
        }
      }
    } else
    for (int32_t it = unit;; it += units) {
      // Every warp takes the same decision, so none is left at a barrier.
      if (!ptx::named_barrier_and(1, 32 * Cfg::kEpiWarps, it < dims.items)) break;
      const FusedItem wi = fused_item<Cfg>(args, dims, it, rank);
      const int buf = acc_iter % Cfg::kAccBufs;
      const uint32_t use_par = static_cast<uint32_t>((acc_iter / Cfg::kAccBufs) & 1);
      ++acc_iter;
      const int32_t row0 = wi.mb * Cfg::kTileM + static_cast<int32_t>(cta) * Cfg::kBM + q * 32;
      const int32_t row = row0 + lane;
      const bool row_in = row < dims.rows;
      // S of a chunk (high and low part; 64 columns each) comes in while the sums
      // do, or while the chunk before is stored (updates of 12 x 512 x 512: 268 us;
      // 292 us with S read when it is needed).
      constexpr bool kSrc = Cfg::kEpi == kEpiSplit || Cfg::kEpi == kEpiSplitSym;
      uint32_t sh[kSrc ? 32 : 1], sl[kSrc ? 32 : 1];
      auto read_source = [&](int c) {
        const int32_t col0 = wi.nb * Cfg::kOutN + c * 64;
        const uint16_t* src = args.src + static_cast<int64_t>(wi.batch) * 2 * args.src_part +
                              static_cast<int64_t>(row) * args.src_ld + col0;
#pragma unroll
        for (int j = 0; j < (kSrc ? 8 : 0); ++j) {
          // Rows of S are padded to a multiple of 8 columns.
          uint4 x = make_uint4(0, 0, 0, 0), y = x;
          if (args.beta != 0.0f && row_in && col0 + j * 8 < args.N) {
            x = ptx::ld_global_v4_u32(src + j * 8);
            y = ptx::ld_global_v4_u32(src + args.src_part + j * 8);
          }
          sh[4 * j] = x.x, sh[4 * j + 1] = x.y, sh[4 * j + 2] = x.z, sh[4 * j + 3] = x.w;
          sl[4 * j] = y.x, sl[4 * j + 1] = y.y, sl[4 * j + 2] = y.z, sl[4 * j + 3] = y.w;
        }
      };
      if constexpr (kSrc) read_source(group);
      int ok = 1;
      if (lane == 0) ok = wait_bar<kPair>(bar_tfull(buf), use_par, w, kSiteTmemFull, it) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ptx::named_barrier_and(1, 32 * Cfg::kEpiWarps, ok != 0)) break;
      ptx::tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(buf * Cfg::kBN);
      auto release_tmem = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            ptx::mbar_arrive_cluster(tempty_bar0 + 8u * buf);
          else
            ptx::mbar_arrive(tempty_bar0 + 8u * buf);
        }
      };
      constexpr int kChunks = Cfg::kOutN / 64;
      if (group >= kChunks) release_tmem();
#pragma unroll 1
      for (int c = group; c < kChunks; c += Cfg::kGroups) {
        const int32_t col0 = wi.nb * Cfg::kOutN + c * 64;
        const bool in = row0 < args.M && col0 < args.N;
        const bool last = c + Cfg::kGroups >= kChunks;
        if constexpr (Cfg::kEpi == kEpiStore) {
          uint32_t v0[32], v1[32], packed[32];
          ptx::tmem_ld_32x32b_x32(t_row + c * 64, v0);
          ptx::tmem_ld_32x32b_x32(t_row + c * 64 + 32, v1);
          ptx::tmem_wait_ld(v0);
          ptx::tmem_regs_ready(v1);
          if (last) release_tmem();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            packed[i] = pack16(bf16, args.alpha * __uint_as_float(v0[2 * i]),
                               args.alpha * __uint_as_float(v0[2 * i + 1]));
            packed[16 + i] = pack16(bf16, args.alpha * __uint_as_float(v1[2 * i]),
                                    args.alpha * __uint_as_float(v1[2 * i + 1]));
          }
          store_chunk(&tmC, packed, col0, row0, wi.batch * args.c_zb, in);
        } else if constexpr (Cfg::kSums) {
          uint32_t v0[32], v1[32];
          ptx::tmem_ld_32x32b_x32(t_row + c * 64, v0);
          ptx::tmem_ld_32x32b_x32(t_row + c * 64 + 32, v1);
          ptx::tmem_wait_ld(v0);
          ptx::tmem_regs_ready(v1);
          if (last) release_tmem();
          if (row0 < dims.rows && col0 < args.N)
            store_sums([&](int i) { return __uint_as_float(i < 32 ? v0[i & 31] : v1[i & 31]); }, col0, row0, row, row_in,
                       wi.batch);
        } else if constexpr (Cfg::kEpi == kEpiGlu) {
          uint32_t h[32], gp[32], up[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t g[32], u[32];
            ptx::tmem_ld_32x32b_x32(t_row + c * 64 + half * 32, g);
            ptx::tmem_ld_32x32b_x32(t_row + Cfg::kOutN + c * 64 + half * 32, u);
            ptx::tmem_wait_ld(g);
            ptx::tmem_regs_ready(u);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float g0 = __uint_as_float(g[2 * i]), g1 = __uint_as_float(g[2 * i + 1]);
              const float u0 = __uint_as_float(u[2 * i]), u1 = __uint_as_float(u[2 * i + 1]);
              h[half * 16 + i] = pack16(bf16, act_value(args.act, g0) * u0, act_value(args.act, g1) * u1);
              gp[half * 16 + i] = pack16(bf16, g0, g1);
              up[half * 16 + i] = pack16(bf16, u0, u1);
            }
          }
          if (last) release_tmem();
          store_chunk(&tmC, h, col0, row0, 0, in);
          if (args.save) {
            store_chunk(&tmD, gp, col0, row0, 0, in);
            store_chunk(&tmD, up, col0, row0, 1, in);
          }
        } else if constexpr (Cfg::kEpi == kEpiGluBwd) {
          uint32_t h[32], dg[32], du[32];
          const uint16_t* gu = args.src + static_cast<int64_t>(row) * args.src_ld + col0;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t v[32], g[16], u[16];
            ptx::tmem_ld_32x32b_x32(t_row + c * 64 + half * 32, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // N is a multiple of 8: a group of eight columns is in or out.
              uint4 a = make_uint4(0, 0, 0, 0), b = a;
              if (row_in && col0 + half * 32 + j * 8 < args.N) {
                a = ptx::ld_global_v4_u32(gu + half * 32 + j * 8);
                b = ptx::ld_global_v4_u32(gu + args.N + half * 32 + j * 8);
              }
              g[4 * j] = a.x, g[4 * j + 1] = a.y, g[4 * j + 2] = a.z, g[4 * j + 3] = a.w;
              u[4 * j] = b.x, u[4 * j + 1] = b.y, u[4 * j + 2] = b.z, u[4 * j + 3] = b.w;
            }
            ptx::tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 gf = unpack16(bf16, g[i]), uf = unpack16(bf16, u[i]);
              const float d0 = __uint_as_float(v[2 * i]), d1 = __uint_as_float(v[2 * i + 1]);
              float a0, a1, s0, s1;
              act_both(args.act, gf.x, a0, s0);
              act_both(args.act, gf.y, a1, s1);
              dg[half * 16 + i] = pack16(bf16, d0 * uf.x * s0, d1 * uf.y * s1);
              du[half * 16 + i] = pack16(bf16, d0 * a0, d1 * a1);
              h[half * 16 + i] = pack16(bf16, a0 * uf.x, a1 * uf.y);
            }
          }
          if (last) release_tmem();
          store_chunk(&tmD, dg, col0, row0, 0, in);
          store_chunk(&tmD, du, col0, row0, 1, in);
          store_chunk(&tmC, h, col0, row0, 0, in);
        } else if constexpr (Cfg::kEpi == kEpiSplit || Cfg::kEpi == kEpiSplitSym) {
          uint32_t hi[32], lo[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t v[32];
            ptx::tmem_ld_32x32b_x32(t_row + c * 64 + half * 32, v);
            if constexpr (Cfg::kParts > 1) {  // from zero, in order, as a cluster adds
              ptx::tmem_wait_ld(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(0.0f + __uint_as_float(v[i]));
#pragma unroll 1
              for (int q = 1; q < Cfg::kParts; ++q) {
                uint32_t u[32];
                ptx::tmem_ld_32x32b_x32(t_row + q * Cfg::kBN + c * 64 + half * 32, u);
                ptx::tmem_wait_ld(u);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
              }
            }
            ptx::tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 xh = unpack16(false, sh[half * 16 + i]), xl = unpack16(false, sl[half * 16 + i]);
              const float r0 = fmaf(args.beta, xh.x + xl.x, args.alpha * __uint_as_float(v[2 * i]));
              const float r1 = fmaf(args.beta, xh.y + xl.y, args.alpha * __uint_as_float(v[2 * i + 1]));
              const uint32_t p = pack16(false, r0, r1);
              const float2 back = unpack16(false, p);
              hi[half * 16 + i] = p;
              lo[half * 16 + i] = pack16(false, r0 - back.x, r1 - back.y);
            }
          }
          if (last)
            release_tmem();
          else
            read_source(c + Cfg::kGroups);
          const int32_t z = wi.batch * args.c_zb;
          store_chunk(&tmC, hi, col0, row0, z, in);
          store_chunk(&tmC, lo, col0, row0, z + 1, in);
          if constexpr (Cfg::kSym) {
            if (wi.mb != wi.nb) {
              store_chunk_t(hi, col0, row0, z, in);
              store_chunk_t(lo, col0, row0, z + 1, in);
            }
          }
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_group<0>();
    __syncwarp();
  }

  if constexpr (Cfg::kSplit > 1) {
    __syncwarp();
    if (!Cfg::kLive || unit < dims.items) {  // (alike in all of the cluster)
      if constexpr (kPair)
        pair_split_epilogue<Cfg>(args, dims, unit, rank, cta, tmem_base, sb + Cfg::kOffEpi, bar_tfull(0), w);
      else
        split_epilogue<Cfg>(args, dims, unit, rank, tmem_base, sb + Cfg::kOffEpi, bar_tfull(0), w);
    }
  }

  ptx::tc_fence_before();
  if constexpr (kPair)
    ptx::cluster_sync();  // neither CTA leaves while the other may touch its memory
  else
    __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<Cfg::kCtas>(tmem_base, Cfg::kTmemCols);
  }
}

}  // namespace ops
}  // namespace gb300
