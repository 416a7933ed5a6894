// norm_kernels.cuh -- layer norm and RMS norm of rows, and their gradients.
//
//   layer norm  m = mean x, v = mean (x - m)^2, r = 1 / sqrt(v + eps), h = (x - m) r
//   RMS norm    r = 1 / sqrt(mean x^2 + eps), h = x r
//   y = h w (+ b)
// and from dy, with q = dy w:
//   dx = r (q - mean q - h mean(q h))        (RMS norm: without mean q)
//   dw = sum over the rows of dy h,  db = sum over the rows of dy
//
// Sums and statistics are fp32.  The mean is taken twice: the second pass sums
// d = x - m1 and d^2 about the first pass's m1, whose rounding (2^-24 m1, which
// a row far from zero shows) c = mean d takes back: m = m1 + c, v = mean d^2 - c^2.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "act.cuh"
#include "ptx_ops.cuh"

namespace gb300 {
namespace ops {

struct NormArgs {
  const void *x, *dy, *weight, *bias;  // weight, bias: null for 1 and 0
  void* y;                             // y, or dx
  float* stats;                        // [T][2]: m, r; RMS norm [T][1]: r; null: not kept
  int64_t ldx, lddy, ldy, T, D;
  float eps;
  float* partial;  // [chunks][2][D]: sums of dy h and of dy over a chunk's rows
  int64_t chunks;
  void *dweight, *dbias;  // null: not wanted
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float* p) { *p = v; }
__device__ __forceinline__ void narrow(float v, __half* p) { *p = __float2half_rn(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// Sums of a and b over the block, the same in every thread; the order is fixed.
// sm: 64 floats, free again after the next barrier.
__device__ __forceinline__ float2 block_sums(float a, float b, float* sm) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    sm[threadIdx.x >> 5] = a;
    sm[32 + (threadIdx.x >> 5)] = b;
  }
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < warps; ++i) s.x += sm[i], s.y += sm[32 + i];
  __syncthreads();
  return s;
}

// kN elements of X as they lie in memory: 16 aligned bytes, or one element.
template <class X, int kN>
struct Vec {
  static_assert(kN * sizeof(X) == 16, "16 bytes");
  uint4 r;
  // Each row is read once: it need not stay in L1, where the weight does.
  __device__ void load(const X* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
  }
  __device__ void get(float (&f)[kN]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(X) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        const float2 v = unpack16(std::is_same<X, __nv_bfloat16>::value, w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    }
  }
  static __device__ void store(X* p, const float (&f)[kN]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(X) == 4)
        w[i] = __float_as_uint(f[i]);
      else
        w[i] = pack16(std::is_same<X, __nv_bfloat16>::value, f[2 * i], f[2 * i + 1]);
    }
    ptx::st_global_v4(p, w[0], w[1], w[2], w[3]);
  }
};
template <class X>
struct Vec<X, 1> {
  X r;
  __device__ void load(const X* p) { r = *p; }
  __device__ void get(float (&f)[1]) const { f[0] = widen(r); }
  static __device__ void store(X* p, const float (&f)[1]) { narrow(f[0], p); }
};

// a + b, a b and a b + c of two pairs at once: the norms of 16-bit rows are bound by
// the instructions they issue, of which these save half.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// The same of kN elements, b and c arrays or one number for all.
__device__ __forceinline__ float2 pair(const float* p, int j) { return make_float2(p[j], p[j + 1]); }
__device__ __forceinline__ float2 pair(float v, int) { return make_float2(v, v); }
__device__ __forceinline__ float single(const float* p) { return p[0]; }
__device__ __forceinline__ float single(float v) { return v; }
template <int kN, class B>
__device__ __forceinline__ void vadd(float (&a)[kN], const B& b) {
  if constexpr (kN == 1) a[0] += single(b);
#pragma unroll
  for (int j = 0; j + 1 < kN; j += 2) {
    const float2 d = add2(pair(a, j), pair(b, j));
    a[j] = d.x, a[j + 1] = d.y;
  }
}
template <int kN, class B>
__device__ __forceinline__ void vmul(float (&a)[kN], const B& b) {
  if constexpr (kN == 1) a[0] *= single(b);
#pragma unroll
  for (int j = 0; j + 1 < kN; j += 2) {
    const float2 d = mul2(pair(a, j), pair(b, j));
    a[j] = d.x, a[j + 1] = d.y;
  }
}
// d = a b + c
template <int kN, class B, class C>
__device__ __forceinline__ void vfma(float (&d)[kN], const float (&a)[kN], const B& b, const C& c) {
  if constexpr (kN == 1) d[0] = fmaf(a[0], single(b), single(c));
#pragma unroll
  for (int j = 0; j + 1 < kN; j += 2) {
    const float2 v = fma2(pair(a, j), pair(b, j), pair(c, j));
    d[j] = v.x, d[j + 1] = v.y;
  }
}
// s += the sum of a, s += the sum of a b
template <int kN>
__device__ __forceinline__ void vsum(float2& s, const float (&a)[kN]) {
  if constexpr (kN == 1) s.x += a[0];
#pragma unroll
  for (int j = 0; j + 1 < kN; j += 2) s = add2(s, pair(a, j));
}
template <int kN>
__device__ __forceinline__ void vdot(float2& s, const float (&a)[kN], const float (&b)[kN]) {
  if constexpr (kN == 1) s.x = fmaf(a[0], b[0], s.x);
#pragma unroll
  for (int j = 0; j + 1 < kN; j += 2) s = fma2(pair(a, j), pair(b, j), s);
}

// kN elements of a weight or bias, which stay in L1.
template <class W, int kN>
__device__ __forceinline__ void load_weight(const W* p, float (&f)[kN]) {
  if constexpr (kN == 1) {
    f[0] = widen(*p);
  } else if constexpr (sizeof(W) == 4) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  } else {
    Vec<W, kN> v;
    v.r = *reinterpret_cast<const uint4*>(p);
    v.get(f);
  }
}

// Sums of a and b over a team of kTeam threads (a warp, or whole warps), the same in
// each and in a fixed order.  sm: 2 x 32 float2 of the team, whose halves alternate
// (turn), so that one barrier between two uses of a half is enough.
template <int kTeam>
__device__ __forceinline__ float2 team_sums(float a, float b, float2* sm, int turn, int team) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  if constexpr (kTeam == 32) return make_float2(a, b);
  constexpr int kWarps = kTeam / 32;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x % kTeam) >> 5;
  float2* half = sm + 32 * turn;
  if (lane == 0) half[warp] = make_float2(a, b);
  ptx::named_barrier_sync(1 + team, kTeam);
  const float2 v = lane < kWarps ? half[lane] : make_float2(0.0f, 0.0f);
  a = v.x, b = v.y;
#pragma unroll
  for (int d = kWarps / 2; d >= 1; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  return make_float2(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, b, 0));
}

// A team of kTeam threads holds a row in registers, kPer vectors of kVec elements a
// thread, and loads its next row before it works on this one.
template <class X, class W, bool kRms, int kVec, int kTeam, int kPer, int kTeams>
__global__ void __launch_bounds__(kTeam* kTeams) norm_rows(const NormArgs a) {
  __shared__ float2 sm[kTeam > 32 ? kTeams * 64 : 1];
  const int team = threadIdx.x / kTeam, at = threadIdx.x % kTeam;
  const int32_t D = static_cast<int32_t>(a.D);
  const X* x = static_cast<const X*>(a.x);
  const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
  const float n = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  Vec<X, kVec> next[kPer];
  auto column = [&](int i) { return (i * kTeam + at) * kVec; };
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) next[i].load(x + row * a.ldx + column(i));
  };
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (t < a.T) load(t);
  for (int turn = 0; t < a.T; t += step) {
    float f[kPer][kVec];
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        next[i].get(f[i]);
        if (!kRms) vsum(s1, f[i]);
      }
    if (t + step < a.T) load(t + step);
    float m1 = 0.0f;
    if constexpr (!kRms) {
      m1 = team_sums<kTeam>(s1.x + s1.y, 0.0f, sm + team * 64, turn, team).x / n;
      turn ^= 1;
      s1 = make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        if (!kRms) {
          vadd(f[i], -m1);
          vsum(s1, f[i]);
        }
        vdot(s2, f[i], f[i]);
      }
    const float2 s = team_sums<kTeam>(s1.x + s1.y, s2.x + s2.y, sm + team * 64, turn, team);
    turn ^= 1;
    const float c = kRms ? 0.0f : s.x / n;
    const float var = s.y / n - c * c;
    const float r = __frsqrt_rn((var < 0.0f ? 0.0f : var) + a.eps);  // (fmaxf would lose a NaN)
    X* y = static_cast<X*>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int col = column(i);
      if (col >= D) continue;
      float g[kVec];
      if (kRms)
        vmul(f[i], r);
      else
        vfma(f[i], f[i], r, -c * r);
      if (w) {
        load_weight<W, kVec>(w + col, g);
        if (!kRms && b) {
          float h[kVec];
          load_weight<W, kVec>(b + col, h);
          vfma(f[i], f[i], g, h);
        } else {
          vmul(f[i], g);
        }
      } else if (!kRms && b) {
        load_weight<W, kVec>(b + col, g);
        vadd(f[i], g);
      }
      Vec<X, kVec>::store(y + col, f[i]);
    }
    if (a.stats && at == 0) {
      if (kRms) {
        a.stats[t] = r;
      } else {
        a.stats[2 * t] = m1 + c;
        a.stats[2 * t + 1] = r;
      }
    }
  }
}

// Rows of norm_rows_back on their way: vectors come through shared memory, of which
// every thread copies and reads its own columns alone (a row ahead in registers keeps
// 32 KB of an SM's loads in flight, three rows ahead 96 KB); single elements through
// registers.
__host__ __device__ constexpr int back_ahead(int threads) { return threads > 512 ? 2 : 3; }
template <class X, int kVec, int kPer>
struct BackRow {
  Vec<X, kVec> x[kPer], g[kPer];
};
template <int kVec, int kPer>
constexpr size_t back_ring(int threads) {
  return kVec > 1 ? static_cast<size_t>(back_ahead(threads) + 1) * 2 * kPer * threads * 16 : 0;
}

// The gradients: teams as above.  A thread's columns are the same in every row, so
// that it keeps their sums of dy h and dy in registers, and their weights; at the end a
// block adds up its teams' sums in order, and leaves one row of `partial`.
template <class X, class W, bool kRms, int kVec, int kTeam, int kPer, int kTeams>
__global__ void __launch_bounds__(kTeam* kTeams, 512 / (kTeam * kTeams) > 0 ? 512 / (kTeam * kTeams) : 1)
    norm_rows_back(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];  // the rows on their way; then sums [2][D], where kTeams > 1
  __shared__ float2 sm[kTeam > 32 ? kTeams * 64 : 1];
  constexpr bool kRing = kVec > 1;
  constexpr int kThreads = kTeam * kTeams, kBackAhead = back_ahead(kThreads), kSlots = kBackAhead + 1;
  // A block of 1024 threads has registers for the sums, and reads the row twice.
  constexpr bool kHold = !kRing || kThreads <= 512;
  const int team = threadIdx.x / kTeam, at = threadIdx.x % kTeam;
  const int32_t D = static_cast<int32_t>(a.D);
  const X *x = static_cast<const X*>(a.x), *dy = static_cast<const X*>(a.dy);
  const W* w = static_cast<const W*>(a.weight);
  const float n = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  BackRow<X, kVec, kPer> next;
  float mn = 0.0f, rn = 0.0f;
  float sw[kPer][kVec] = {}, sb[kRms ? 1 : kPer][kVec] = {}, wv[kHold ? kPer : 1][kVec];
  auto column = [&](int i) { return (i * kTeam + at) * kVec; };
  // Slot s, vector i of x (which = 0) or dy (1) of this thread.
  const uint32_t mine = ptx::smem_addr(ring) + threadIdx.x * 16;
  auto slot = [&](int s, int which, int i) {
    return mine + static_cast<uint32_t>(((s * 2 + which) * kPer + i) * kThreads) * 16u;
  };
  auto fetch = [&](int64_t row, int s) {
    if (row < a.T) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (column(i) < D) {
          if constexpr (kRing) {
            ptx::cp_async_16(slot(s, 0, i), x + row * a.ldx + column(i));
            ptx::cp_async_16(slot(s, 1, i), dy + row * a.lddy + column(i));
          } else {
            next.x[i].load(x + row * a.ldx + column(i));
            next.g[i].load(dy + row * a.lddy + column(i));
          }
        }
    }
    if constexpr (kRing) ptx::cp_async_commit();
  };
  auto stats = [&](int64_t row) {
    if (row < a.T) {
      if (!kRms) mn = a.stats[2 * row];
      rn = a.stats[kRms ? row : 2 * row + 1];
    }
  };
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  for (int s = 0; s < (kRing ? kBackAhead : 1); ++s) fetch(t + s * step, s);
  stats(t);
  auto weights = [&](int i, float(&v)[kVec]) {
    if (w && column(i) < D) {
      load_weight<W, kVec>(w + column(i), v);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = 1.0f;
    }
  };
#pragma unroll
  for (int i = 0; i < (kHold ? kPer : 0); ++i) weights(i, wv[i]);
  // h and q of vector i, and dy.
  auto work_out = [&](int i, float m, float r, float(&h)[kVec], float(&q)[kVec], float(&g)[kVec]) {
    next.x[i].get(h);
    next.g[i].get(g);
    if (!kRms) vadd(h, -m);
    vmul(h, r);
#pragma unroll
    for (int j = 0; j < kVec; ++j) q[j] = g[j];
    if constexpr (!kHold) weights(i, wv[0]);
    vmul(q, wv[kHold ? i : 0]);
  };
  int at_slot = 0;
  for (int turn = 0; t < a.T; t += step, turn ^= 1) {
    const float m = mn, r = rn;
    float h[kHold ? kPer : 1][kVec], q[kHold ? kPer : 1][kVec], g[kVec];
    const int here = at_slot;
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
    if constexpr (kRing) {
      ptx::cp_async_wait<kBackAhead - 1>();
      const int free_slot = at_slot == 0 ? kSlots - 1 : at_slot - 1;  // read in the turn before
      fetch(t + kBackAhead * step, free_slot);
      at_slot = at_slot + 1 == kSlots ? 0 : at_slot + 1;
    }
    stats(t + step);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        if constexpr (kRing) {
          next.x[i].r = ptx::ld_shared_v4_u32(slot(here, 0, i));
          next.g[i].r = ptx::ld_shared_v4_u32(slot(here, 1, i));
        }
        const int k = kHold ? i : 0;
        work_out(i, m, r, h[k], q[k], g);
        vfma(sw[i], g, h[k], sw[i]);
        if (!kRms) vadd(sb[kRms ? 0 : i], g);
        if (!kRms) vsum(s1, q[k]);
        vdot(s2, q[k], h[k]);
      }
    if constexpr (!kRing) fetch(t + step, 0);
    const float2 s = team_sums<kTeam>(s1.x + s1.y, s2.x + s2.y, sm + team * 64, turn, team);
    const float c1 = kRms ? 0.0f : s.x / n, c2 = s.y / n;
    X* dx = static_cast<X*>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        const int k = kHold ? i : 0;
        if constexpr (!kHold) {
          next.x[i].r = ptx::ld_shared_v4_u32(slot(here, 0, i));
          next.g[i].r = ptx::ld_shared_v4_u32(slot(here, 1, i));
          work_out(i, m, r, h[k], q[k], g);
        }
        if (!kRms) vadd(q[k], -c1);
        vfma(q[k], h[k], -c2, q[k]);
        vmul(q[k], r);
        Vec<X, kVec>::store(dx + column(i), q[k]);
      }
  }
  if constexpr (kRing) {
    ptx::cp_async_wait<0>();
    if (kTeams > 1) __syncthreads();  // the sums take the ring's place
  }
  float* sums = reinterpret_cast<float*>(ring);
  if (!a.partial) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * D;
#pragma unroll 1
  for (int k = 0; k < kTeams; ++k) {
    if (team == k) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int col = column(i);
        if (col >= D) continue;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          float vw = sw[i][j], vb = kRms ? 0.0f : sb[kRms ? 0 : i][j];
          if (k > 0) vw += sums[col + j], vb += sums[D + col + j];
          float* to = k + 1 < kTeams ? sums : out;
          to[col + j] = vw;
          if (!kRms) to[D + col + j] = vb;
        }
      }
    }
    if (kTeams > 1) __syncthreads();
  }
}

// One block per row, element by element: rows of any length, start and distance.
template <class X, class W, bool kRms>
__global__ void __launch_bounds__(512) norm_any(const NormArgs a) {
  __shared__ float sm[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const X* x = static_cast<const X*>(a.x) + t * a.ldx;
  X* y = static_cast<X*>(a.y) + t * a.ldy;
  const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
  const float n = static_cast<float>(a.D);
  float m1 = 0.0f;
  if (!kRms) {
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) s += widen(x[i]);
    m1 = block_sums(s, 0.0f, sm).x / n;
  }
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    const float d = widen(x[i]) - m1;
    s1 += d;
    s2 = fmaf(d, d, s2);
  }
  const float2 s = block_sums(s1, s2, sm);
  const float c = kRms ? 0.0f : s.x / n;
  const float v = s.y / n - c * c;
  const float r = __frsqrt_rn((v < 0.0f ? 0.0f : v) + a.eps);  // (fmaxf would lose a NaN)
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    float v = ((widen(x[i]) - m1) - c) * r;
    if (w) v *= widen(w[i]);
    if (b) v += widen(b[i]);
    narrow(v, y + i);
  }
  if (a.stats && threadIdx.x == 0) {
    if (kRms) {
      a.stats[t] = r;
    } else {
      a.stats[2 * t] = m1 + c;
      a.stats[2 * t + 1] = r;
    }
  }
}

template <class X, class W, bool kRms>
__global__ void __launch_bounds__(512) norm_dx_any(const NormArgs a) {
  __shared__ float sm[64];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const X *x = static_cast<const X*>(a.x) + t * a.ldx, *dy = static_cast<const X*>(a.dy) + t * a.lddy;
  X* dx = static_cast<X*>(a.y) + t * a.ldy;
  const W* w = static_cast<const W*>(a.weight);
  const float n = static_cast<float>(a.D);
  const float m = kRms ? 0.0f : a.stats[2 * t], r = kRms ? a.stats[t] : a.stats[2 * t + 1];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    const float h = (widen(x[i]) - m) * r, q = widen(dy[i]) * (w ? widen(w[i]) : 1.0f);
    s1 += q;
    s2 = fmaf(q, h, s2);
  }
  const float2 s = block_sums(s1, s2, sm);
  const float c1 = kRms ? 0.0f : s.x / n, c2 = s.y / n;
  for (int64_t i = threadIdx.x; i < a.D; i += blockDim.x) {
    const float h = (widen(x[i]) - m) * r, q = widen(dy[i]) * (w ? widen(w[i]) : 1.0f);
    narrow(r * ((q - c1) - h * c2), dx + i);
  }
}

// grid (columns / 32, chunks), block 32 x 8: sums of dy h and dy over a chunk.
template <class X, bool kRms>
__global__ void __launch_bounds__(256) norm_dw_any(const NormArgs a) {
  __shared__ float sm[2][8][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t t0 = blockIdx.y * a.T / a.chunks, t1 = (blockIdx.y + 1) * a.T / a.chunks;
  const X *x = static_cast<const X*>(a.x) + col, *dy = static_cast<const X*>(a.dy) + col;
  float sw = 0.0f, sb = 0.0f;
  if (col < a.D)
    for (int64_t t = t0 + warp; t < t1; t += 8) {
      const float m = kRms ? 0.0f : a.stats[2 * t], r = kRms ? a.stats[t] : a.stats[2 * t + 1];
      const float g = widen(dy[t * a.lddy]);
      sw = fmaf(g, (widen(x[t * a.ldx]) - m) * r, sw);
      sb += g;
    }
  sm[0][warp][lane] = sw;
  sm[1][warp][lane] = sb;
  __syncthreads();
  if (warp < 2 && col < a.D) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[warp][i][lane];
    a.partial[(2 * static_cast<int64_t>(blockIdx.y) + warp) * a.D + col] = s;
  }
}

// The sums of all chunks: 32 columns by 16 groups of chunks, each in order, then the
// groups in order.  grid (columns / 32, weight or bias).
template <class W>
__global__ void __launch_bounds__(512) norm_dw_sum(const NormArgs a) {
  __shared__ float sm[16][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  W* out = static_cast<W*>(blockIdx.y == 0 ? a.dweight : a.dbias);
  if (!out) return;
  float s = 0.0f;
  if (col < a.D) {
#pragma unroll 8
    for (int64_t c = group; c < a.chunks; c += 16) s += a.partial[(2 * c + blockIdx.y) * a.D + col];
  }
  sm[group][lane] = s;
  __syncthreads();
  if (group == 0 && col < a.D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += sm[i][lane];
    narrow(s, out + col);
  }
}

}  // namespace ops
}  // namespace gb300
