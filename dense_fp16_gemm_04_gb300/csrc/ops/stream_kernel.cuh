// stream_kernel.cuh -- products of a few tokens with a weight matrix read
// once:  y[t, n] = sum_k x[t, k] W[n, k]  for T <= 16 tokens, W in 16 bits or
// in 4 bits with a scale (and a zero point) per group of a row:
//
//   W[n, k] = s[n, k / G] (q[n, k] - z[n, k / G]),   q, z in 0 .. 15.
//
// Bound by the weights' bytes.  The sums run on warp-level matrix products
// (16 rows of W x 16 k x 8 tokens): tcgen05 would have to stage every weight
// through shared memory for a tile of 64 rows or more, while here a warp's
// weights go from memory to registers and stop there, 16 bytes a lane, in the
// order a row stores them.  That order is free because a sum over k may be
// taken in any order, the same for W and x: lane t of a row's four lanes takes
// eight consecutive k of every 32 as its k-slots of two products.
//
// 4-bit codes become 16-bit floats without a conversion: a code's bits below
// the exponent of 1024 (fp16) or 128 (bf16) read 1024 + q or 128 + q, and
// subtracting 1024 + z or 128 + z is exact.  Products of 16-bit x and these
// integers are exact in fp32; the scale multiplies the fp32 sum of its group.
//
// A CTA takes 16 rows of the output (gated: the 16 gate rows and 16 up rows
// of the same columns), its warps split K, and their sums meet in shared
// memory in warp order (the result does not depend on timing).
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
  int32_t T, N, K;       // N: rows of the output per matrix (gated: W has 2N rows)
  int32_t group_shift;   // log2 G
  int32_t act;
};

constexpr int kStreamMaxWarps = 16;

// The quad's 4 x 4 transpose: lane t holds word j of row j' = t; afterwards
// it holds word t of every lane's: v[j] = lane j's word t.
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[4], int t) {
  const bool hi = (t & 2) != 0, odd = (t & 1) != 0;
  {
    const uint32_t s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 2), r1 = __shfl_xor_sync(0xffffffffu, s1, 2);
    if (hi)
      v[0] = r0, v[1] = r1;
    else
      v[2] = r0, v[3] = r1;
  }
  {
    const uint32_t s0 = odd ? v[0] : v[1], s1 = odd ? v[2] : v[3];
    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, s0, 1), r1 = __shfl_xor_sync(0xffffffffu, s1, 1);
    if (odd)
      v[0] = r0, v[2] = r1;
    else
      v[1] = r0, v[3] = r1;
  }
}

// Eight codes to four pairs (code j, code j + 4), less the zero point.
template <bool kBf16>
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t zsub, uint32_t (&p)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | (kBf16 ? 0x43004300u : 0x64006400u);
    if constexpr (kBf16) {
      const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                       *reinterpret_cast<const __nv_bfloat162*>(&zsub));
      p[j] = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v),
                                *reinterpret_cast<const __half2*>(&zsub));
      p[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

// (1024 + z, 1024 + z) or (128 + z, 128 + z).
template <bool kBf16>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  const uint32_t v = (kBf16 ? 0x4300u : 0x6400u) | z;
  return v | (v << 16);
}

// kMT: 16-row tiles per warp (2 when gated: gate rows, up rows); kNT: tiles of
// 8 tokens.
template <bool kBf16, bool kW4, bool kGlu, int kNT>
__global__ void __launch_bounds__(32 * kStreamMaxWarps) stream_kernel(const StreamArgs a) {
  constexpr int kMT = kGlu ? 2 : 1;
  extern __shared__ float red[];  // [warp][kMT][kNT][4][32]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int32_t n0 = blockIdx.x * 16;
  const int32_t t0 = blockIdx.y * (8 * kNT);
  // This warp's k-range, in units of 128 k.
  const int32_t units = (a.K + 127) / 128;
  const int32_t u0 = static_cast<int32_t>(static_cast<int64_t>(warp) * units / warps);
  const int32_t u1 = static_cast<int32_t>(static_cast<int64_t>(warp + 1) * units / warps);
  float acc[kMT][kNT][4];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
  // Rows of W this lane reads: g and g + 8 of each tile; rows past N read the
  // last row (their sums are not stored).
  int64_t row[kMT][2];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int32_t n = n0 + g + 8 * r;
      row[m][r] = static_cast<int64_t>(n < a.N ? n : a.N - 1) + static_cast<int64_t>(m) * a.N;
    }
  // Tokens this lane supplies: t0 + g of each tile.
  const uint16_t* xp[kNT];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const int32_t tok = t0 + 8 * n + g;
    xp[n] = tok < a.T ? a.x + static_cast<int64_t>(tok) * a.ldx : nullptr;
  }
  auto load_x = [&](int n, int32_t k) {
    return xp[n] != nullptr && k < a.K ? ptx::ld_global_v4_u32(xp[n] + k) : make_uint4(0, 0, 0, 0);
  };
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if constexpr (kW4) {
    const uint8_t* w = static_cast<const uint8_t*>(a.w);
    const int64_t groups = a.K >> a.group_shift;
    for (int32_t u = u0; u < u1; ++u) {
      const int32_t k0 = u * 128;
      uint32_t c[kMT][2][4];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 v = k0 + 32 * t < a.K
                              ? ptx::ld_global_stream_v4(w + row[m][r] * a.ldw + k0 / 2 + 16 * t)
                              : make_uint4(0, 0, 0, 0);
          c[m][r][0] = v.x, c[m][r][1] = v.y, c[m][r][2] = v.z, c[m][r][3] = v.w;
        }
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) quad_transpose(c[m][r], t);
      float part[kMT][kNT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t k = k0 + 32 * j;
        if (k >= a.K) break;
        const int32_t grp = k >> a.group_shift;
        const bool first = ((k >> 5) & ((1 << (a.group_shift - 5)) - 1)) == 0 || j == 0;
        const bool last = (((k + 32) >> 5) & ((1 << (a.group_shift - 5)) - 1)) == 0 || j == 3 || k + 32 >= a.K;
        uint32_t xb[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const uint4 v = load_x(n, k + 8 * t);
          xb[n][0] = __byte_perm(v.x, v.z, 0x5410);
          xb[n][1] = __byte_perm(v.x, v.z, 0x7632);
          xb[n][2] = __byte_perm(v.y, v.w, 0x5410);
          xb[n][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
          uint32_t p[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t z = a.zeros ? a.zeros[row[m][r] * groups + grp] & 15u : 8u;
            dequant8<kBf16>(c[m][r][j], zero_pair<kBf16>(z), p[r]);
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            if (first)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[m][n][i] = 0.0f;
            ptx::mma_16816<kBf16>(part[m][n], p[0][0], p[1][0], p[0][1], p[1][1], xb[n][0], xb[n][1]);
            ptx::mma_16816<kBf16>(part[m][n], p[0][2], p[1][2], p[0][3], p[1][3], xb[n][2], xb[n][3]);
          }
          if (last) {
            const float s0 = widen16(kBf16, a.scales[row[m][0] * groups + grp]);
            const float s1 = widen16(kBf16, a.scales[row[m][1] * groups + grp]);
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              acc[m][n][0] = fmaf(s0, part[m][n][0], acc[m][n][0]);
              acc[m][n][1] = fmaf(s0, part[m][n][1], acc[m][n][1]);
              acc[m][n][2] = fmaf(s1, part[m][n][2], acc[m][n][2]);
              acc[m][n][3] = fmaf(s1, part[m][n][3], acc[m][n][3]);
            }
          }
        }
      }
    }
  } else {
    const uint16_t* w = static_cast<const uint16_t*>(a.w);
    for (int32_t u = u0; u < u1; ++u) {
      uint4 wv[4][kMT][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t k = u * 128 + 32 * j + 8 * t;
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            wv[j][m][r] = k < a.K ? ptx::ld_global_stream_v4(w + row[m][r] * a.ldw + k)
                                  : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const uint4 x = load_x(n, u * 128 + 32 * j + 8 * t);
#pragma unroll
          for (int m = 0; m < kMT; ++m) {
            const uint4 p = wv[j][m][0], q = wv[j][m][1];
            ptx::mma_16816<kBf16>(acc[m][n], p.x, q.x, p.y, q.y, x.x, x.y);
            ptx::mma_16816<kBf16>(acc[m][n], p.z, q.z, p.w, q.w, x.z, x.w);
          }
        }
      }
    }
  }
  // Sum the warps' k-ranges, in order.
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[((warp * kMT + m) * kNT + n) * 128 + i * 32 + lane] = acc[m][n][i];
  __syncthreads();
  // Thread j finishes element (row, token) of the CTA's 16 x 8 kNT tile.
  for (int e = threadIdx.x; e < 16 * 8 * kNT; e += blockDim.x) {
    const int r = e & 15, tok = e >> 4;
    const int32_t n = n0 + r, tk = t0 + tok;
    if (n >= a.N || tk >= a.T) continue;
    // Fragment element of (row r, token tok & 7): lane 4 (r & 7) + (tok & 7) / 2,
    // value (tok & 1) + 2 (r >= 8).
    const int nt = tok >> 3, c = tok & 7;
    const int at = ((c & 1) + 2 * (r >> 3)) * 32 + 4 * (r & 7) + (c >> 1);
    float v[kMT];
#pragma unroll
    for (int m = 0; m < kMT; ++m) {
      float s = 0.0f;
      for (int wp = 0; wp < warps; ++wp) s += red[((wp * kMT + m) * kNT + nt) * 128 + at];
      v[m] = s;
    }
    float out = v[0];
    if constexpr (kGlu) {
      out = act_value(a.act, v[0]) * v[1];
      if (a.gu) {
        a.gu[static_cast<int64_t>(tk) * 2 * a.N + n] = round16(kBf16, v[0]);
        a.gu[static_cast<int64_t>(tk) * 2 * a.N + a.N + n] = round16(kBf16, v[1]);
      }
    }
    a.y[static_cast<int64_t>(tk) * a.ldy + n] = round16(kBf16, out);
  }
}

}  // namespace ops
}  // namespace gb300
