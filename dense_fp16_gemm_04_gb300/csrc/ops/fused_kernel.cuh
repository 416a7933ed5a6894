// fused_kernel.cuh -- products with fused epilogues on the tensor cores
// (tcgen05) of sm_103a: the matrix work of the gated feed-forward block, of
// its backward pass and of the orthogonalised update.
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
//   kEpiPartial  fp32 partial sums of one of several k-ranges of a tile, to be
//                added by a second kernel (fused_reduce.cuh): for few tiles
//                with long K.
//
// Units (a CTA with a 128-row tile, or a pair of CTAs with a 256-row one) are
// persistent and take tiles round robin.  Inside a CTA: warp 0 loads A and
// warp 6 loads B (TMA, 128-byte swizzle, a ring of kStages k-blocks), warp 1
// issues tcgen05.mma, warps 2-5 run the epilogue of the tile before (the
// accumulator is double-buffered in TMEM).  Bounded waits as in
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
  kEpiPartial = 5,
};

struct FusedArgs {
  int32_t M, N;               // rows and columns of the output (of h for the gated forward)
  int32_t tiles_m, tiles_n;   // tiles of one matrix of the batch
  int32_t per_batch;          // tiles computed per matrix (tiles_m tiles_n, or the triangle)
  int32_t items;              // work items: per_batch x batch x splits
  int32_t splits;             // k-ranges per tile (kEpiPartial), else 1
  int32_t num_kb;             // 64-deep k-blocks of one segment
  int32_t segs;               // segments (1, or 3: high high + high low + low high)
  int32_t z_mul;              // third coordinate of matrix b of the batch: b z_mul + part
  int32_t group_m;            // raster group height, in tiles
  int32_t a_mn, b_mn;         // operand layouts: 0 K-contiguous, 1 MN-contiguous
  int32_t bf16;               // operands and 16-bit outputs are bf16
  int32_t act, save;          // gated epilogues: activation; keep g and u
  float alpha, beta;
  const uint16_t* src;        // kEpiSplit*: S (rows src_ld apart), its low part src_part further,
  int64_t src_ld, src_part;   //   the next matrix of the batch 2 src_part further;
                              // kEpiGluBwd: g and u, [M, 2N]
  float* partial;             // kEpiPartial: [split][M][part_ld]
  int64_t part_ld, part_stride;
  uint32_t* err;
  uint64_t timeout_ns;
  int32_t skip_kb;            // fault injection, -1 = off
};

template <int kCtas_, int kBN_, int kStages_, int kEpi_, int kEpiBufs_>
struct FusedCfg {
  static constexpr int kCtas = kCtas_;
  static constexpr int kBN = kBN_;  // columns of the accumulator
  static constexpr int kStages = kStages_;
  static constexpr int kEpi = kEpi_;
  static constexpr int kEpiBufs = kEpiBufs_;  // 32 x 64 staging buffers per epilogue warp
  static constexpr bool kGlu = kEpi == kEpiGlu;
  static constexpr bool kSym = kEpi == kEpiSplitSym;
  static constexpr int kOutN = kGlu ? kBN / 2 : kBN;  // output columns per tile
  static constexpr int kBM = 128, kBK = 64;
  static constexpr int kTileM = kBM * kCtas;
  static constexpr int kBRows = kBN / kCtas;
  static constexpr int kABytes = kBM * kBK * 2;
  static constexpr int kBBytes = kBRows * kBK * 2;
  static constexpr int kEpiWarps = 4;
  static constexpr int kBufBytes = 32 * 128;
  static constexpr int kOffA = 0;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffEpi = kOffB + kStages * kBBytes;
  static constexpr int kOffBar = kOffEpi + kEpiWarps * kEpiBufs * kBufBytes;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int kOffSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffSlot + 4;
  static constexpr int kSmemBytes = kOffAbort + 4 + 1024;  // + slack to align the base
  static constexpr int kTmemCols = 2 * kBN;
  static constexpr int kThreads = 256;
  static constexpr uint32_t kIdesc = ptx::idesc_f16(kTileM, kBN, true);
  static_assert(kSmemBytes <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(kOutN % 64 == 0, "the epilogue works on 64-column chunks");
  static_assert(!kSym || kTileM == kBN, "symmetric tiles are square");
  static_assert(kTmemCols <= 512, "TMEM columns");
};

// One tile's k-range.
struct FusedItem {
  int32_t mb, nb, batch, split, kb0, kb1;
};

template <class Cfg>
__device__ __forceinline__ FusedItem fused_item(const FusedArgs& a, int32_t it) {
  FusedItem w;
  const int32_t total = a.num_kb * a.segs;
  int32_t t = it;
  w.split = 0;
  if constexpr (Cfg::kEpi == kEpiPartial) {
    // Neighbouring units take the k-ranges of one tile.
    t = it / a.splits;
    w.split = it - t * a.splits;
  }
  w.kb0 = static_cast<int32_t>(static_cast<int64_t>(w.split) * total / a.splits);
  w.kb1 = static_cast<int32_t>(static_cast<int64_t>(w.split + 1) * total / a.splits);
  w.batch = t / a.per_batch;
  const int32_t r = t - w.batch * a.per_batch;
  if constexpr (Cfg::kSym) {
    // Triangle r: column nb holds rows 0 .. nb.
    int32_t j = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
    while ((j + 1) * (j + 2) / 2 <= r) ++j;
    while (j * (j + 1) / 2 > r) --j;
    w.nb = j;
    w.mb = r - j * (j + 1) / 2;
  } else {
    raster(r, a.tiles_m, a.tiles_n, a.group_m, w.mb, w.nb);
  }
  return w;
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    fused_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD,
                 const FusedArgs args) {
  constexpr int S = Cfg::kStages;
  constexpr bool kPair = Cfg::kCtas == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = kPair ? ptx::cluster_ctarank() : 0u;  // 0: issues the MMAs
  const int32_t unit = kPair ? static_cast<int32_t>(ptx::cluster_id_x()) : static_cast<int32_t>(blockIdx.x);
  const int32_t units = kPair ? static_cast<int32_t>(ptx::num_clusters_x()) : static_cast<int32_t>(gridDim.x);

  const uint32_t bar0 = sb + Cfg::kOffBar;
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto bar_tfull = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto bar_tempty = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
  const uint32_t bar_mma_done = bar0 + 8u * (2 * S + 4);
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
      ptx::mbar_init(bar_tempty(b), Cfg::kEpiWarps * Cfg::kCtas);
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
  if constexpr (kPair)
    ptx::cluster_sync();  // both CTAs' barriers exist before either uses the other's
  else
    __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffSlot);

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------- TMA producers --
    const bool is_a = warp == 0;
    const CUtensorMap* tm = is_a ? &tmA : &tmB;
    const bool mn = is_a ? args.a_mn != 0 : args.b_mn != 0;
    const uint32_t op_bytes = is_a ? Cfg::kABytes : Cfg::kBBytes;
    const uint32_t op_base = sb + (is_a ? Cfg::kOffA : Cfg::kOffB);
    const uint32_t op_tx = op_bytes * Cfg::kCtas;
    // The operand's rows arrive as kBoxes boxes per stage.  Gated forward, B:
    // the gate rows and up rows of the same columns of h (a pair's CTAs load
    // one half each, a lone CTA both); then the row and the matrix differ.
    constexpr int kGluBoxes = kPair ? 1 : 2;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int stage = 0;
    uint32_t phase = 0;
    int64_t fills = 0;
    bool ok = true, first_item = true;
    for (int32_t it = unit; ok && it < args.items; it += units) {
      const FusedItem wi = fused_item<Cfg>(args, it);
      int32_t row, z0 = wi.batch * args.z_mul;
      if (is_a)
        row = wi.mb * Cfg::kTileM + static_cast<int32_t>(cta) * Cfg::kBM;
      else if (Cfg::kGlu)
        row = wi.nb * Cfg::kOutN;
      else
        row = wi.nb * Cfg::kBN + static_cast<int32_t>(cta) * Cfg::kBRows;
      int32_t seg = wi.kb0 / args.num_kb, k = wi.kb0 - seg * args.num_kb;
      for (int32_t kb = wi.kb0; kb < wi.kb1; ++kb) {
        if (!wait_bar_warp<kPair>(bar_empty(stage), phase ^ 1u, w, kSiteEmpty, it)) {
          ok = false;
          break;
        }
        const bool skip = args.skip_kb == kb && first_item && unit == 0 && cta == 0;
        if (!skip && ptx::elect_one()) {
          const uint32_t dst = op_base + static_cast<uint32_t>(stage) * op_bytes;
          // Segments: high high, high low, low high.
          const int32_t z = z0 + (is_a ? (seg == 2 ? 1 : 0) : (seg == 1 ? 1 : 0));
          uint32_t full = bar_full(stage);
          if constexpr (kPair) {
            full = ptx::mapa(full, 0);
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
        if (++k == args.num_kb) {
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
      const uint64_t b_desc0 = args.b_mn ? ptx::sw128_mnmajor_desc(sb + Cfg::kOffB)
                                         : ptx::sw128_kmajor_desc(sb + Cfg::kOffB);
      constexpr uint64_t kADescStage = Cfg::kABytes >> 4;
      constexpr uint64_t kBDescStage = Cfg::kBBytes >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int32_t acc_iter = 0;
      bool ok = true;
      for (int32_t it = unit; ok && it < args.items; it += units) {
        const FusedItem wi = fused_item<Cfg>(args, it);
        const int buf = acc_iter & 1;
        const uint32_t use_par = static_cast<uint32_t>((acc_iter >> 1) & 1);
        if (!wait_bar_warp<kPair>(bar_tempty(buf), use_par ^ 1u, w, kSiteTmemEmpty, it)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * Cfg::kBN);
        for (int32_t kb = wi.kb0; kb < wi.kb1; ++kb) {
          if (!wait_bar_warp<kPair>(bar_full(stage), phase, w, kSiteFull, it)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t a_desc = a_desc0 + kADescStage * static_cast<uint32_t>(stage);
          const uint64_t b_desc = b_desc0 + kBDescStage * static_cast<uint32_t>(stage);
          const uint32_t acc_first = kb != wi.kb0 ? 1u : 0u;
          if (ptx::elect_one()) {
#pragma unroll
            for (int k = 0; k < Cfg::kBK / 16; ++k)
              ptx::mma_f16<Cfg::kCtas>(d_tmem, a_desc + a_kstep * k, b_desc + b_kstep * k, idesc,
                                       k != 0 ? 1u : acc_first);
            if constexpr (kPair)
              ptx::mma_commit_pair(bar_empty(stage), 0x3);
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
            ptx::mma_commit_pair(bar_tfull(buf), 0x3);
          else
            ptx::mma_commit(bar_tfull(buf));
        }
        __syncwarp();
        ++acc_iter;
      }
      // Every MMA has finished before tensor memory is freed.
      if (ptx::elect_one()) {
        if constexpr (kPair)
          ptx::mma_commit_pair(bar_mma_done, 0x1);
        else
          ptx::mma_commit(bar_mma_done);
      }
      __syncwarp();
      wait_bar_warp<kPair>(bar_mma_done, 0u, w, kSiteMmaDone, -1, /*honor_abort=*/false);
    }
  } else if (warp >= 2 && warp < 2 + Cfg::kEpiWarps) {
    // ------------------------------------------------------------ epilogue --
    ptx::griddep_wait();  // reads S, g and u; writes the outputs
    const int q = warp & 3;  // this warp may touch TMEM lanes 32q .. 32q+31 only
    const uint32_t stage_base =
        sb + Cfg::kOffEpi + static_cast<uint32_t>(q * Cfg::kEpiBufs * Cfg::kBufBytes);
    const uint32_t tempty_bar0 = kPair ? ptx::mapa(bar_tempty(0), 0) : bar_tempty(0);
    const bool bf16 = args.bf16 != 0;
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
    // A 32 x 64 chunk (row `lane`, columns packed in pairs) through a swizzled
    // buffer to rows row0.., columns col0.. of matrix z.  Every buffer taken
    // commits one group, empty where nothing of the chunk is in range, so that
    // the count in take_buf holds.
    auto store_chunk = [&](const CUtensorMap* m, const uint32_t (&packed)[32], int32_t col0,
                           int32_t row0, int32_t z, bool in) {
      const uint32_t sbuf = take_buf();
      const uint32_t row_addr = sbuf + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        ptx::st_shared_v4(row_addr + ((static_cast<uint32_t>(j) ^ (lane & 7u)) << 4), packed[4 * j],
                          packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (in) ptx::tma_store_3d(m, sbuf, col0, row0, z);
        ptx::bulk_commit_group();
      }
    };
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
    for (int32_t it = unit;; it += units) {
      // Every warp takes the same decision, so none is left at a barrier.
      if (!ptx::named_barrier_and(1, 32 * Cfg::kEpiWarps, it < args.items)) break;
      const FusedItem wi = fused_item<Cfg>(args, it);
      const int buf = acc_iter & 1;
      const uint32_t use_par = static_cast<uint32_t>((acc_iter >> 1) & 1);
      ++acc_iter;
      int ok = 1;
      if (lane == 0) ok = wait_bar<kPair>(bar_tfull(buf), use_par, w, kSiteTmemFull, it) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ptx::named_barrier_and(1, 32 * Cfg::kEpiWarps, ok != 0)) break;
      ptx::tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(buf * Cfg::kBN);
      const int32_t row0 = wi.mb * Cfg::kTileM + static_cast<int32_t>(cta) * Cfg::kBM + q * 32;
      const int32_t row = row0 + lane;
      const bool row_in = row < args.M;
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
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int32_t col0 = wi.nb * Cfg::kOutN + c * 64;
        const bool in = row0 < args.M && col0 < args.N;
        const bool last = c == kChunks - 1;
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
          store_chunk(&tmC, packed, col0, row0, wi.batch * args.z_mul, in);
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
          const bool with_src = args.beta != 0.0f;
          const uint16_t* sh = args.src + static_cast<int64_t>(wi.batch) * 2 * args.src_part +
                               static_cast<int64_t>(row) * args.src_ld + col0;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t v[32], a[16], b[16];
            ptx::tmem_ld_32x32b_x32(t_row + c * 64 + half * 32, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // Rows of S are padded to a multiple of 8 columns.
              uint4 x = make_uint4(0, 0, 0, 0), y = x;
              if (with_src && row_in && col0 + half * 32 + j * 8 < args.N) {
                x = ptx::ld_global_v4_u32(sh + half * 32 + j * 8);
                y = ptx::ld_global_v4_u32(sh + args.src_part + half * 32 + j * 8);
              }
              a[4 * j] = x.x, a[4 * j + 1] = x.y, a[4 * j + 2] = x.z, a[4 * j + 3] = x.w;
              b[4 * j] = y.x, b[4 * j + 1] = y.y, b[4 * j + 2] = y.z, b[4 * j + 3] = y.w;
            }
            ptx::tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 xh = unpack16(false, a[i]), xl = unpack16(false, b[i]);
              const float r0 = fmaf(args.beta, xh.x + xl.x, args.alpha * __uint_as_float(v[2 * i]));
              const float r1 = fmaf(args.beta, xh.y + xl.y, args.alpha * __uint_as_float(v[2 * i + 1]));
              const uint32_t p = pack16(false, r0, r1);
              const float2 back = unpack16(false, p);
              hi[half * 16 + i] = p;
              lo[half * 16 + i] = pack16(false, r0 - back.x, r1 - back.y);
            }
          }
          if (last) release_tmem();
          const int32_t z = wi.batch * args.z_mul;
          store_chunk(&tmC, hi, col0, row0, z, in);
          store_chunk(&tmC, lo, col0, row0, z + 1, in);
          if constexpr (Cfg::kSym) {
            if (wi.mb != wi.nb) {
              store_chunk_t(hi, col0, row0, z, in);
              store_chunk_t(lo, col0, row0, z + 1, in);
            }
          }
        } else {  // kEpiPartial
          float* out = args.partial + static_cast<int64_t>(wi.split) * args.part_stride +
                       static_cast<int64_t>(row) * args.part_ld + col0;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t v[32];
            ptx::tmem_ld_32x32b_x32(t_row + c * 64 + half * 32, v);
            ptx::tmem_wait_ld(v);
            if (last && half == 1) release_tmem();
#pragma unroll
            for (int j = 0; j < 8; ++j)  // part_ld is a multiple of 4 and covers N
              if (row_in && col0 + half * 32 + j * 4 < args.N)
                ptx::st_global_v4(out + half * 32 + j * 4, v[4 * j], v[4 * j + 1], v[4 * j + 2],
                                  v[4 * j + 3]);
          }
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_group<0>();
    __syncwarp();
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
