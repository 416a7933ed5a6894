// stream_kernel.cuh -- products of a few tokens with a weight matrix read
// once:  y[t, n] = sum_k x[t, k] W[n, k]  for up to 16 tokens at a time, W in 16
// bits or in 4 bits with a scale (and a zero point) per group of a row:
//
//   W[n, k] = s[n, k / G] (q[n, k] - z[n, k / G]),   q, z in 0 .. 15.
//
// The least it can take is the weights' bytes.  16-bit weights come close
// (8192 x 16384 gated block, one token: 123 us, 96% of a copy's bandwidth); 4-bit
// ones are bound by the instructions that unpack them (one token x 16384 gated
// columns x 8192, groups of 32: 37 us for 151 MB, 60%; 303 instructions per warp
// for 32 rows x 128 k, of which 96 unpack and 24 multiply, at 1.9 per clock).
//
// The sums run on warp-level matrix products (16 rows of W x 16 k x 8 tokens):
// tcgen05 would have to stage every weight through shared memory for a tile of
// 64 rows or more, while here a warp's weights are read by the lane that fetched
// them, 16 bytes a lane, in the order a row stores them.  That order is free
// because a sum over k may be taken in any order, the same for W and x: lane t of
// a row's four lanes takes eight consecutive k of every 32 as its k-slots of two
// products.
//
// 4-bit codes become 16-bit floats without a conversion: four bits set in the
// mantissa of 64 (fp16) or 128 (bf16) read O + q with O that number.  With
//
//   sum over a group of (q - z) x = sum (O + q) x - (O + z) sum x,
//
// nothing is subtracted from the codes; the group's sum of x comes from one
// product more, of a matrix of ones with the same x.  Products of 16-bit x and
// O + q are exact; the offset makes the fp32 sum's roundings at most 16 to 30
// times those of q x alone, 2^-20 of the group's size, far below the 16-bit
// result's own rounding.  The scale multiplies the finished fp32 sum.  A sum that
// does not come out finite is taken again product by product (direct_sum).
//
// A lane's 16 bytes are 32 codes of one row, so the four lanes of a row hold
// 128 k: one group, two, or four.  Smaller groups are kept apart in one of two
// ways.  In turn: the four lanes read a group's codes from shared memory together
// (8 or 4 bytes a lane of what another lane fetched), so that a product sums one
// group alone.  By columns, for as many tokens as fit: a product's eight columns
// are 4 or 2 tokens x 2 or 4 groups, and a column's x is zero in the lanes whose k
// lie in another group.  Columns cost fewer instructions while one tile of them
// holds the tokens, and twice or four times the products beyond.
//
// CTAs are persistent: x (this CTA's k-slice of it) is staged in shared memory
// once, and tiles of 32 rows of W follow one another (gated: 16 gate rows and
// the 16 up rows of the same columns), two products for every read of x: with
// 16 rows the reads of x alone filled shared memory's bandwidth.  A tile's
// k-blocks are dealt to the warps in turn, so that the CTA reads contiguous
// pieces of each row; every lane keeps its pieces of the next `ring` blocks in
// flight (asynchronous copies to shared memory: no barrier, no registers), across
// tile ends.  The warps' sums meet in shared memory in warp order, so the result
// does not depend on timing.  Where there are few tiles, or x does not fit, K is
// also cut over CTAs and a second kernel adds the slices.
#pragma once
#include "act.cuh"
#include "ptx_ops.cuh"

namespace gb300 {
namespace ops {

struct StreamArgs {
  const uint16_t* x;     // [T, K], rows ldx apart
  int64_t ldx;
  const void* w;         // 16-bit [rows, K] or codes [rows, K / 2], rows ldw elements (bytes) apart
  int64_t ldw;
  const uint16_t* scales;  // [rows, K / G]
  const uint8_t* zeros;    // [rows, K / G] or null (8)
  uint16_t* y;           // [T, N], rows ldy apart
  int64_t ldy;
  uint16_t* gu;          // gated: g and u, [T, 2N], or null
  float* partial;        // several k-slices: [slice][T][N or 2N]
  int32_t T, N, K;       // N: columns of the output this launch makes, of `cols` in all
  int32_t cols;
  int64_t up_w, up_s;    // gated: from gate to up rows, in bytes of W and in scales
  int32_t group_shift;   // log2 G
  int32_t act;
  int32_t ring;          // blocks a warp keeps in flight, 2 .. 4
  int32_t early;         // W may be read before the previous kernel has ended
};

constexpr int kStreamMaxWarps = 16;

// How W is stored: 16-bit values, or codes whose groups are 32, 64, or 128 k
// and more; the small ones kept apart in turn or (Few) by columns.
enum StreamW : int { kW16 = 0, kW4G32 = 1, kW4G64 = 2, kW4G128 = 3, kW4G32Few = 4, kW4G64Few = 5 };

// k of a block; its groups that share a product's columns, and that take turns;
// tokens of an 8-column tile.
__host__ __device__ constexpr int stream_block_k(int w) { return w == kW16 ? 32 : 128; }
__host__ __device__ constexpr int stream_groups(int w) { return w == kW4G32Few ? 4 : w == kW4G64Few ? 2 : 1; }
__host__ __device__ constexpr int stream_turns(int w) { return w == kW4G32 ? 4 : w == kW4G64 ? 2 : 1; }
__host__ __device__ constexpr int stream_tokens(int w) { return 8 / stream_groups(w); }
// Rows of W a lane reads per tile (g, g + 8 of two 16-row halves); what a warp
// keeps for a block in flight: 16 bytes of W a row and lane and, with codes,
// 8 bytes a row for its scales and 8 for its zero points.
constexpr int kStreamRows = 4;
__host__ __device__ constexpr int stream_slot_bytes(int w) {
  return kStreamRows * (32 * 16 + (w == kW16 ? 0 : 8 * 16));
}
constexpr int kStreamMaxRing = 4;
constexpr int kStreamHead = 128 + 16;  // of x in shared memory
__host__ __device__ constexpr int stream_tile(bool glu) { return glu ? 16 : 32; }  // columns of y

// Eight codes to four pairs (code j, code j + 4) of O + q: a shift and one
// and-or each.
template <bool kBf16>
__device__ __forceinline__ void offset_codes(uint32_t w, uint32_t (&p)[4]) {
  constexpr uint32_t bits = kBf16 ? 0x43004300u : 0x54005400u;
  if constexpr (kBf16) {
    p[0] = ptx::and_or<0x000f000fu>(w, bits);
    p[1] = ptx::and_or<0x000f000fu>(w >> 4, bits);
    p[2] = ptx::and_or<0x000f000fu>(w >> 8, bits);
    p[3] = ptx::and_or<0x000f000fu>(w >> 12, bits);
  } else {
    const uint32_t w8 = w >> 8;  // shifts left run on another pipe than the bit operations
    p[0] = ptx::and_or<0x00f000f0u>(w << 4, bits);
    p[1] = ptx::and_or<0x00f000f0u>(w, bits);
    p[2] = ptx::and_or<0x00f000f0u>(w8 << 4, bits);
    p[3] = ptx::and_or<0x00f000f0u>(w8, bits);
  }
}

// The aligned 4-byte word that holds *p.
__device__ __forceinline__ const void* word_of(const void* p) {
  return reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(3));
}

// Token tk's sum with row n of W (gated: of half m) over k0 <= k < k1 (multiples
// of 32), product by product as the formula has it.
template <bool kBf16>
__device__ __forceinline__ float direct_sum(const StreamArgs& a, int32_t tk, int32_t n, int32_t m, int32_t k0,
                                            int32_t k1) {
  const int64_t groups = a.K >> a.group_shift, row = m * a.up_s + n * groups;
  const uint16_t* const x = a.x + tk * a.ldx;
  const uint8_t* const codes = static_cast<const uint8_t*>(a.w) + m * a.up_w + n * a.ldw;
  float sum = 0.0f;
#pragma unroll 1
  for (int32_t k = k0; k < k1; k += 8) {
    const int64_t j = row + (k >> a.group_shift);
    const float scale = widen16(kBf16, a.scales[j]);
    const int32_t zero = a.zeros ? a.zeros[j] : 8;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (k >> 1));
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const int32_t q = static_cast<int32_t>(w >> (4 * i) & 15) - zero;
      sum = fmaf(scale * static_cast<float>(q), widen16(kBf16, x[k + i]), sum);
    }
  }
  return sum;
}

template <bool kBf16>
__device__ __noinline__ float direct_sum_call(const StreamArgs& a, int32_t tk, int32_t n, int32_t m, int32_t k0,
                                              int32_t k1) {
  return direct_sum<kBf16>(a, tk, n, m, k0, k1);
}

template <bool kBf16, int kW, bool kGlu, int kNT>
__global__ void __launch_bounds__(32 * kStreamMaxWarps, 1) stream_kernel(const StreamArgs a) {
  constexpr bool kW4 = kW != kW16;
  constexpr int kMT = 2;  // 16-row halves of a tile
  constexpr int kBK = stream_block_k(kW);
  constexpr int kSlot = stream_slot_bytes(kW);
  constexpr int kRows = kStreamRows;
  constexpr int kTileN = stream_tile(kGlu);
  constexpr int kGroups = stream_groups(kW);
  constexpr int kTurns = stream_turns(kW);
  constexpr int kInBlock = kGroups * kTurns;  // groups of a block
  constexpr int kTok = stream_tokens(kW);  // tokens per 8-column tile
  constexpr int kRed = kMT * kNT * 128;    // floats one warp leaves per tile
  extern __shared__ __align__(16) uint8_t stream_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int32_t t0 = blockIdx.z * (kTok * kNT);
  const int32_t tokens = min(a.T - t0, kTok * kNT);
  // This CTA's k-slice (whole blocks; slices partition them).
  const int32_t blocks = (a.K + kBK - 1) / kBK;
  const int32_t b0 = static_cast<int32_t>(static_cast<int64_t>(blockIdx.y) * blocks / gridDim.y);
  const int32_t b1 = static_cast<int32_t>(static_cast<int64_t>(blockIdx.y + 1) * blocks / gridDim.y);
  const int32_t k_begin = b0 * kBK;
  float* const red0 = reinterpret_cast<float*>(stream_smem);  // [2][warp][kMT][kNT][row][column]
  float* red = red0;
  // [warp][slot]: [row of the lane][lane][16 B], then the scales and the zero
  // points [row][g][two words].
  uint8_t* wr = reinterpret_cast<uint8_t*>(red0 + 2 * warps * kRed);
  uint8_t* xs = wr + warps * a.ring * kSlot;  // kStreamHead bytes (zeros, then ones), then [block][i][token][t][16 B]
  const int32_t per_tile = (b1 - b0 - warp + warps - 1) / warps;  // this warp's blocks of a tile
  const int32_t tiles = (a.N + kTileN - 1) / kTileN;
  const int32_t my_tiles = (tiles - static_cast<int32_t>(blockIdx.x) + static_cast<int32_t>(gridDim.x) - 1) /
                           static_cast<int32_t>(gridDim.x);

  // The warp's blocks in order: block load_blk of tile load_tile.  A lane reads
  // rows i = 0 .. 3: g and g + 8 of the tile's first half, then of its second.
  // row_of(tile, i): the row of W, from the base of its half (32-bit byte
  // offsets: the host cuts larger matrices).  Rows past N read the last row,
  // and k past K the last codes: the sums of the former are not stored, x is 0
  // in the latter.
  int32_t load_tile = blockIdx.x, load_blk = 0, to_load = my_tiles * per_tile;
  const uint32_t slot0 = ptx::smem_addr(wr) + warp * (a.ring * kSlot);
  const uint32_t groups = kW4 ? a.K >> a.group_shift : 0;
  const uint32_t row_bytes = static_cast<uint32_t>(a.ldw) * (kW4 ? 1 : 2);
  constexpr int kOwn = kGlu ? 2 : 4;  // different rows (gated: the up rows repeat the gate's)
  auto row_of = [&](int32_t tile, int i) {
    return static_cast<uint32_t>(min(tile * kTileN + g + 8 * i, a.N - 1));
  };
  uint32_t w_off[kOwn], s_off = 0;  // s_off: of row i = t, whose scales this lane fetches
  auto rows_of_tile = [&]() {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) w_off[i] = row_of(load_tile, i) * row_bytes;
    if constexpr (kW4) s_off = row_of(load_tile, t & (kOwn - 1)) * groups;
  };
  rows_of_tile();
  const uint8_t* w_base[2] = {static_cast<const uint8_t*>(a.w), static_cast<const uint8_t*>(a.w) + a.up_w};
  const uint16_t* s_base[2] = {a.scales, a.scales + a.up_s};
  const uint8_t* z_base[2] = {a.zeros, a.zeros + a.up_s};
  constexpr int kHalf = kGlu ? 1 : 0;  // whether rows 2, 3 have the other base
  // The low bits of those addresses: where in its word a scale or zero lies.
  const uint32_t s_low[2] = {static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_base[0])),
                             static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_base[1]))};
  const uint32_t z_low[2] = {static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z_base[0])),
                             static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z_base[1]))};
  uint32_t sum_off[kOwn];  // rows times groups, of the tile being summed
#pragma unroll
  for (int i = 0; i < kOwn; ++i) sum_off[i] = row_of(load_tile, i) * groups;
  // The scales of a row's groups in one block share an aligned word (of 8 bytes
  // for four), and so do its zero points, unless rows do not hold whole blocks
  // or start off such a word: then they are read when they are needed.  Lane t
  // fetches row t's: 32 rows with one instruction.
  const bool words = kInBlock == 1 || (((groups | static_cast<uint32_t>(a.up_s)) & (kInBlock - 1)) == 0 &&
                                       (reinterpret_cast<uintptr_t>(a.scales) & (2 * kInBlock - 1)) == 0 &&
                                       (reinterpret_cast<uintptr_t>(a.zeros) & (kInBlock - 1)) == 0);
  const uint16_t* s_mine = kGlu && t > 1 ? s_base[1] : s_base[0];
  const uint8_t* z_mine = kGlu && t > 1 ? z_base[1] : z_base[0];
  // The first group of block b, or of pair `pair` of its groups.
  auto group_of = [&](int32_t b, int pair) {
    return static_cast<uint32_t>(b * kBK >> a.group_shift) + (2u * pair & (kInBlock - 1));
  };
  // Where a lane's 16 bytes of a row go: with groups in turn, the other lanes of
  // the row read parts of them, and chunks change places so that the eight rows
  // of such a read fall on different banks.
  const uint32_t swap = kTurns > 1 ? (g & 2) | (g >> 2) : 0;
  const uint32_t put = (g * 4 + (t ^ swap)) * 16;
  auto issue = [&](uint32_t slot) {
    const int32_t b = b0 + load_blk * warps + warp;
    const int32_t k0 = b * kBK;
    const uint32_t at = kW4 ? min(k0 + 32 * t, a.K - 32) >> 1 : 2 * min(k0 + 8 * t, a.K - 8);
    const uint32_t bytes = k0 + 8 * t < a.K ? 16 : 0;  // zeros past K: infinity times x's 0 is NaN
    const uint32_t dst = slot + put;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const void* src = w_base[kHalf * (i >> 1)] + (w_off[i & (kOwn - 1)] + at);
      if constexpr (kW4)
        ptx::cp_async_16(dst + i * 512, src);
      else
        ptx::cp_async_16(dst + i * 512, src, bytes);
    }
    if constexpr (kW4) {
      if (words) {  // the aligned word lies in the same allocation
        const uint32_t at = s_off + group_of(b, 0), dst = slot + kRows * 512 + t * 64 + g * 8;
        if constexpr (kInBlock == 4)
          ptx::cp_async_8(dst, s_mine + at);
        else
          ptx::cp_async_4(dst, word_of(s_mine + at));
        if (a.zeros) ptx::cp_async_4(dst + kRows * 64, word_of(z_mine + at));
      }
    }
    --to_load;
    if (++load_blk == per_tile) {
      load_blk = 0;
      load_tile += gridDim.x;
      rows_of_tile();
    }
  };

  if (!a.early) ptx::griddep_wait();
  for (int i = 0; i < a.ring; ++i) {
    if (to_load > 0) issue(slot0 + i * kSlot);
    ptx::cp_async_commit();
  }
  if (a.early) ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // Stage x: 16-byte chunks of eight k, in the order the products read them
  // (4 bits: chunk 4 t + i of a block is word i of lane t), four loads in
  // flight a thread; zeros past K.
  {
    constexpr int kPer = kBK / 8;  // chunks per block
    const int32_t chunks = (b1 - b0) * kPer;
    if (threadIdx.x < 36) reinterpret_cast<uint32_t*>(xs)[threadIdx.x] = threadIdx.x < 32 ? 0u : kBf16 ? 0x3f803f80u : 0x3c003c00u;
    int32_t next_tok = 0, next_c = threadIdx.x;  // chunk next_c of token next_tok
    while (next_tok < tokens) {
      uint4 v[4];
      int32_t tok[4], c[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        while (next_c >= chunks) {
          next_c -= chunks;
          ++next_tok;
        }
        tok[u] = next_tok;
        c[u] = next_c;
        next_c += blockDim.x;
        v[u] = make_uint4(0, 0, 0, 0);
        if (tok[u] < tokens && k_begin + 8 * c[u] < a.K)
          v[u] = ptx::ld_global_v4_u32(a.x + (t0 + tok[u]) * a.ldx + k_begin + 8 * c[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (tok[u] >= tokens) break;
        const int32_t blk = c[u] / kPer, ch = c[u] & (kPer - 1);
        uint4 o = v[u];
        if constexpr (kW4)  // pairs (x j, x j + 4), as the codes unpack
          o = make_uint4(__byte_perm(v[u].x, v[u].z, 0x5410), __byte_perm(v[u].x, v[u].z, 0x7632),
                         __byte_perm(v[u].y, v[u].w, 0x5410), __byte_perm(v[u].y, v[u].w, 0x7632));
        // The product i and lane l that take this chunk.
        const int i = kTurns == 4 ? ch >> 2 : kTurns == 2 ? (ch >> 3) * 2 + (ch & 1) : kW4 ? ch & 3 : 0;
        const int l = kTurns == 4 ? ch & 3 : kTurns == 2 ? ch >> 1 & 3 : kW4 ? ch >> 2 : ch;
        *reinterpret_cast<uint4*>(xs + kStreamHead + (((blk * (kPer / 4) + i) * tokens + tok[u]) * 4 + l) * 16) = o;
      }
    }
  }
  __syncthreads();
  // Column g of tile n is token n kTok + g / kGroups, group g % kGroups; lane
  // t's k lie in group t kGroups / 4 of the block.
  uint32_t xl[kNT], x_step[kNT];  // bytes from i to i + 1; the other lanes stay at the zeros
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const int32_t tok = n * kTok + g / kGroups;
    const bool mine = tok < tokens && t * kGroups / 4 == g % kGroups;
    xl[n] = ptx::smem_addr(xs) + (mine ? kStreamHead + tok * 64 + t * 16 : lane % 8 * 16);
    x_step[n] = mine ? tokens * 64 : 0;
  }

  float acc[kMT][kNT][4];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
  int32_t tile = blockIdx.x;
  // The matrix of ones, from shared memory: the compiler makes a constant anew
  // for every product.  (Four groups and two tiles have no registers to hold it.)
  constexpr uint32_t kOnes = kBf16 ? 0x3f803f80u : 0x3c003c00u;
  uint4 ones = make_uint4(kOnes, kOnes, kOnes, kOnes);
  if constexpr (kW4 && kTurns * kNT < 8) ones = ptx::ld_shared_v4_u32(ptx::smem_addr(xs) + 128);
  auto consume = [&](uint32_t slot, int32_t rel) {  // block b0 + rel
    constexpr int kWords = kBK / 32;
    uint32_t xa[kNT];
#pragma unroll
    for (int n = 0; n < kNT; ++n) xa[n] = xl[n] + rel * kWords * x_step[n];
    // Word i of a row holds the codes of product i.
    uint32_t wv[kRows][4];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (kTurns == 1) {
        const uint4 v = ptx::ld_shared_v4_u32(slot + i * 512 + put);
        wv[i][0] = v.x, wv[i][1] = v.y, wv[i][2] = v.z, wv[i][3] = v.w;
      } else if constexpr (kTurns == 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint2 v = ptx::ld_shared_v2_u32(slot + i * 512 + g * 64 + ((2 * s + (t >> 1)) ^ swap) * 16 + (t & 1) * 8);
          wv[i][2 * s] = v.x, wv[i][2 * s + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) wv[i][s] = ptx::ld_shared_u32(slot + i * 512 + g * 64 + (s ^ swap) * 16 + t * 4);
      }
    }
    if constexpr (kW4) {
      // Scales (two to a word) and zero points (two bytes) of a pair of groups.
      constexpr int kPairs = kTurns == 4 ? 2 : 1;
      uint32_t sv[kPairs][kRows], zv[kPairs][kRows];
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const int pair = kGroups > 1 ? t : p;
        const uint32_t j = group_of(b0 + rel, pair), at = slot + kRows * 512 + g * 8;
        if (words) {
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            sv[p][i] = ptx::ld_shared_u32(at + i * 64 + (kInBlock == 4 ? (pair & 1) * 4 : 0));
            // A lone scale is the word's low or high half.
            if (kInBlock == 1) sv[p][i] >>= ((s_low[kHalf * (i >> 1)] + 2 * (sum_off[i & (kOwn - 1)] + j)) & 2) * 8;
          }
          if (a.zeros) {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
              zv[p][i] = ptx::ld_shared_u32(at + (kRows + i) * 64) >>
                         ((z_low[kHalf * (i >> 1)] + sum_off[i & (kOwn - 1)] + j) & 3) * 8;
          }
        } else {
          const uint32_t j0 = min(j, groups - 1), j1 = min(j0 + 1, groups - 1);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const uint32_t o = sum_off[i & (kOwn - 1)];
            const uint16_t* sp = s_base[kHalf * (i >> 1)] + o;
            const uint8_t* zp = z_base[kHalf * (i >> 1)] + o;
            sv[p][i] = sp[j0] | static_cast<uint32_t>(sp[j1]) << 16;
            if (a.zeros) zv[p][i] = zp[j0] | static_cast<uint32_t>(zp[j1]) << 8;
          }
        }
      }
      // -(O + z) is z's bits in the mantissa of -O.
      float z0[kPairs][kRows], z1[kPairs][kRows];
      constexpr uint32_t kMinusO = kBf16 ? 0xc3000000u : 0xc2800000u;
      constexpr int kBit = kBf16 ? 16 : 17;
      if (a.zeros) {
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            z0[p][i] = __uint_as_float(ptx::and_or<15u << kBit>(zv[p][i] << kBit, kMinusO));
            z1[p][i] = kInBlock > 1 ? __uint_as_float(ptx::and_or<15u << kBit>(zv[p][i] << (kBit - 8), kMinusO))
                                    : z0[p][i];
          }
      } else {
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
#pragma unroll
          for (int i = 0; i < kRows; ++i) z0[p][i] = z1[p][i] = __uint_as_float(kMinusO | 8u << kBit);
      }
      float part[kMT][kNT][4], sx[kNT][4];  // sums of (O + q) x, and of x (in every row)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const bool first = i % (kWords / kTurns) == 0;  // of a group's, or of the block's
        uint4 xb[kNT];
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          xb[n] = ptx::ld_shared_v4_u32(xa[n]);
          xa[n] += x_step[n];
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          if (first)
            ptx::mma_16816_zero<kBf16>(sx[n], ones.x, ones.y, ones.z, ones.w, xb[n].x, xb[n].y);
          else
            ptx::mma_16816<kBf16>(sx[n], ones.x, ones.y, ones.z, ones.w, xb[n].x, xb[n].y);
          ptx::mma_16816<kBf16>(sx[n], ones.x, ones.y, ones.z, ones.w, xb[n].z, xb[n].w);
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          uint32_t p0[4], p1[4];
          offset_codes<kBf16>(wv[2 * m][i], p0);
          offset_codes<kBf16>(wv[2 * m + 1][i], p1);
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            if (first)
              ptx::mma_16816_zero<kBf16>(part[m][n], p0[0], p1[0], p0[1], p1[1], xb[n].x, xb[n].y);
            else
              ptx::mma_16816<kBf16>(part[m][n], p0[0], p1[0], p0[1], p1[1], xb[n].x, xb[n].y);
            ptx::mma_16816<kBf16>(part[m][n], p0[2], p1[2], p0[3], p1[3], xb[n].z, xb[n].w);
          }
        }
        if ((i + 1) % (kWords / kTurns) != 0) continue;
        // The end of a group (by columns: of the groups of this lane's two).
        const int turn = i / (kWords / kTurns), pair = turn / 2;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float2 f = unpack16(kBf16, sv[pair][r]);
          const float f0 = turn & 1 ? f.y : f.x, f1 = kGroups > 1 ? f.y : f0;
          const float m0 = turn & 1 ? z1[pair][r] : z0[pair][r], m1 = kGroups > 1 ? z1[pair][r] : m0;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            float* c = acc[r >> 1][n] + 2 * (r & 1);
            const float* p = part[r >> 1][n] + 2 * (r & 1);
            c[0] = fmaf(f0, fmaf(m0, sx[n][0], p[0]), c[0]);
            c[1] = fmaf(f1, fmaf(m1, sx[n][1], p[1]), c[1]);
          }
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const uint4 x = ptx::ld_shared_v4_u32(xa[n]);
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          const uint32_t *p = wv[2 * m], *q = wv[2 * m + 1];
          ptx::mma_16816<kBf16>(acc[m][n], p[0], q[0], p[1], q[1], x.x, x.y);
          ptx::mma_16816<kBf16>(acc[m][n], p[2], q[2], p[3], q[3], x.z, x.w);
        }
      }
    }
  };

  auto finish_tile = [&]() {
    // The warps' sums, in warp order.  Two tiles' places take turns: a thread
    // that passes a tile's barrier has read the sums of the one before.
    red = red0 + (red == red0 ? warps * kRed : 0);
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        float* p = red + warp * kRed + (m * kNT + n) * 128 + g * 8 + 2 * t;
        *reinterpret_cast<float2*>(p) = make_float2(acc[m][n][0], acc[m][n][1]);
        *reinterpret_cast<float2*>(p + 64) = make_float2(acc[m][n][2], acc[m][n][3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      }
    __syncthreads();
    // A thread per element (gated: of both halves); then the columns of one
    // token.
    constexpr int kEach = kGlu ? 2 : 1;
    for (int e = threadIdx.x; e < 2 / kEach * 128 * kNT; e += blockDim.x) {
      float v[kEach];
#pragma unroll
      for (int m = 0; m < kEach; ++m) {
        float s = 0.0f;
#pragma unroll 4
        for (int w = 0; w < warps; ++w) s += red[w * kRed + m * kNT * 128 + e];
#pragma unroll
        for (int d = 1; d < kGroups; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        v[m] = s;
      }
      const int col = e & 7, q = e >> 7;  // q: 16-row half (plain) and column tile
      const int tok = q % kNT * kTok + col / kGroups;
      const int32_t n = tile * kTileN + q / kNT * 16 + ((e >> 3) & 15), tk = t0 + tok;
      if (n >= a.N || tok >= tokens || col % kGroups != 0) continue;
      if constexpr (kW4) {
        // An infinite x, or one whose products with O + q overflow, leaves infinity
        // less infinity where the formula has a signed infinity or a finite sum.
        // Inline or as a call by what the loop over blocks keeps in registers: plain
        // products of 9 to 16 tokens, groups of 64 (fp16, 16 x 8192 x 8192), 27.6 us
        // inline and 23.4 as a call; of 128 22.0 and 22.7; one token (4096 x 4096,
        // groups of 128) 4.3 and 4.8.
        constexpr auto sum = kNT == 2 && !kGlu && kTurns > 1 ? direct_sum_call<kBf16> : direct_sum<kBf16>;
        const int32_t k_end = min(b1 * kBK, a.K);
#pragma unroll
        for (int m = 0; m < kEach; ++m)
          if (!isfinite(v[m])) v[m] = sum(a, tk, n, m, k_begin, k_end);
      }
      if (gridDim.y > 1) {
#pragma unroll
        for (int m = 0; m < kEach; ++m)
          a.partial[((static_cast<int64_t>(blockIdx.y) * a.T + tk) * kEach + m) * a.N + n] = v[m];
        continue;
      }
      float out = v[0];
      if constexpr (kGlu) {
        out = act_value(a.act, v[0]) * v[1];
        if (a.gu) {
          a.gu[static_cast<int64_t>(tk) * 2 * a.cols + n] = round16(kBf16, v[0]);
          a.gu[static_cast<int64_t>(tk) * 2 * a.cols + a.cols + n] = round16(kBf16, v[1]);
        }
      }
      a.y[static_cast<int64_t>(tk) * a.ldy + n] = round16(kBf16, out);
    }
    tile += gridDim.x;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) sum_off[i] = row_of(tile, i) * groups;
  };
  uint32_t slot = slot0;
#pragma unroll 1
  for (int32_t i = 0; i < my_tiles; ++i) {
#pragma unroll 1
    for (int32_t rel = warp; rel < b1 - b0; rel += warps) {
      // This lane's oldest block has landed; then the warp's, whose lanes share
      // the scales.
      if (a.ring == 4)
        ptx::cp_async_wait<3>();
      else if (a.ring == 3)
        ptx::cp_async_wait<2>();
      else
        ptx::cp_async_wait<1>();
      __syncwarp();
      consume(slot, rel);
      __syncwarp();
      if (to_load > 0) issue(slot);
      ptx::cp_async_commit();  // one group per block, empty at the end
      slot += kSlot;
      if (slot == slot0 + a.ring * kSlot) slot = slot0;
    }
    finish_tile();
  }
}

// Adds the k-slices of stream_kernel, in order, and finishes the output.
template <bool kGlu>
__global__ void __launch_bounds__(256) stream_reduce(const StreamArgs a, int32_t slices, int32_t bf16) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  constexpr int kMT = kGlu ? 2 : 1;
  const int64_t total = static_cast<int64_t>(a.T) * a.N, stride = total * kMT;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t tk = i / a.N, n = i - tk * a.N;
    const float* p = a.partial + tk * kMT * a.N + n;
    float v[kMT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) v[m] = 0.0f;
    for (int32_t s = 0; s < slices; ++s)
#pragma unroll
      for (int m = 0; m < kMT; ++m) v[m] += __ldcg(p + s * stride + m * a.N);
    float out = v[0];
    if constexpr (kGlu) {
      out = act_value(a.act, v[0]) * v[1];
      if (a.gu) {
        a.gu[tk * 2 * a.cols + n] = round16(bf16, v[0]);
        a.gu[tk * 2 * a.cols + a.cols + n] = round16(bf16, v[1]);
      }
    }
    a.y[tk * a.ldy + n] = round16(bf16, out);
  }
}

}  // namespace ops
}  // namespace gb300
