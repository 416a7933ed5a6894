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

// Two fp32 numbers in a pair of registers, with add, multiply and fused multiply-add
// of both at once: two in one issue slot, at the rate of two single ones (layer norm
// backward of 8192 x 8192 bf16 77 us, with single ones 80).  The same names for one
// number.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ f32x2 vadd(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 vmul(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 vfma(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(f32x2 v) {
  const float2 f = unpack2(v);
  return f.x + f.y;
}
__device__ __forceinline__ float total(float v) { return v; }

// kN elements of X: as they lie in memory, 16 or 4 aligned bytes or one element (Vec),
// and as fp32 numbers, in kW pairs or as one (Reg).
template <int kN>
struct Reg {
  typedef f32x2 E;
  static constexpr int kW = kN / 2;
  E v[kW];
  static __device__ E all(float f) { return pack2(f, f); }
};
template <>
struct Reg<1> {
  typedef float E;
  static constexpr int kW = 1;
  E v[1];
  static __device__ E all(float f) { return f; }
};

template <class X, int kN>
struct Vec {
  static_assert(kN * sizeof(X) == 16, "16 bytes");
  static constexpr int kBytes = 16;
  uint4 r;
  __device__ void load_shared(uint32_t addr) { r = ptx::ld_shared_v4_u32(addr); }
  // Each row is read once: it need not stay in L1, where the weight does.
  __device__ void load(const X* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
  }
  __device__ void get(Reg<kN>& f) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) f.v[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<X, __nv_bfloat16>::value) {
          // bf16 is the upper half of an fp32 (two instructions; the conversion takes three).
          f.v[i] = pack2(__uint_as_float(__byte_perm(w[i], 0, 0x1044)), __uint_as_float(w[i] & 0xffff0000u));
        } else {
          const float2 v = unpack16(false, w[i]);
          f.v[i] = pack2(v.x, v.y);
        }
      }
    }
  }
  static __device__ void store(X* p, const Reg<kN>& f) {
    uint32_t w[4];
    if constexpr (sizeof(X) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 v = unpack2(f.v[i]);
        w[2 * i] = __float_as_uint(v.x), w[2 * i + 1] = __float_as_uint(v.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2(f.v[i]);
        w[i] = pack16(std::is_same<X, __nv_bfloat16>::value, v.x, v.y);
      }
    }
    ptx::st_global_v4(p, w[0], w[1], w[2], w[3]);
  }
};
template <class X>
struct Vec<X, 2> {
  static_assert(sizeof(X) == 2, "4 bytes");
  static constexpr int kBytes = 4;
  uint32_t r;
  __device__ void load(const X* p) { r = *reinterpret_cast<const uint32_t*>(p); }
  __device__ void load_shared(uint32_t addr) { r = ptx::ld_shared_u32(addr); }
  __device__ void get(Reg<2>& f) const {
    const float2 v = unpack16(std::is_same<X, __nv_bfloat16>::value, r);
    f.v[0] = pack2(v.x, v.y);
  }
  static __device__ void store(X* p, const Reg<2>& f) {
    const float2 v = unpack2(f.v[0]);
    *reinterpret_cast<uint32_t*>(p) = pack16(std::is_same<X, __nv_bfloat16>::value, v.x, v.y);
  }
};
template <class X>
struct Vec<X, 1> {
  X r;
  __device__ void load(const X* p) { r = *p; }
  __device__ void get(Reg<1>& f) const { f.v[0] = widen(r); }
  static __device__ void store(X* p, const Reg<1>& f) { narrow(f.v[0], p); }
};

// kN elements of a weight or bias, which stay in L1.
template <class W, int kN>
__device__ __forceinline__ void load_weight(const W* p, Reg<kN>& f) {
  if constexpr (kN == 1) {
    f.v[0] = widen(*p);
  } else if constexpr (kN == 2) {  // (which may start on any element)
    f.v[0] = pack2(widen(p[0]), widen(p[1]));
  } else if constexpr (sizeof(W) == 4) {
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f.v[i / 2] = pack2(v.x, v.y), f.v[i / 2 + 1] = pack2(v.z, v.w);
    }
  } else {
    Vec<W, kN> v;
    v.r = *reinterpret_cast<const uint4*>(p);
    v.get(f);
  }
}

// Sums of two numbers over a team of kTeam threads (a warp, or whole warps), the same
// in each and in a fixed order: add() by every thread, ready() before get().  sm: 128
// floats of the team, whose halves are for turns 0 and 1: with one ready() between a
// half's get() and its next add(), one barrier a turn is enough.
template <int kTeam>
struct TeamSums {
  static constexpr int kWarps = kTeam / 32;
  float *sm, held;  // a warp's own: a in its lower half, b in the upper
  int team;
  __device__ TeamSums(float* sm, int team) : sm(sm), held(0.0f), team(team) {}
  __device__ void add(float2 v, int turn) {
    const int lane = threadIdx.x & 31;
    const bool low = lane < 16;
    float s = low ? v.x : v.y;
    s += __shfl_xor_sync(0xffffffffu, low ? v.y : v.x, 16);
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if constexpr (kWarps == 1)
      held = s;
    else if ((lane & 15) == 0)
      sm[64 * turn + 2 * lane + (threadIdx.x % kTeam) / 32] = s;
  }
  __device__ void ready() {
    if constexpr (kWarps > 1) ptx::named_barrier_sync(1 + team, kTeam);
  }
  __device__ float2 get(int turn) {
    float s = held;
    if constexpr (kWarps > 1) {
      constexpr int kHalf = kWarps > 16 ? 16 : kWarps;  // a lane takes one warp's, or two
      const float* from = sm + 64 * turn + 2 * (threadIdx.x & 16);
      s = from[threadIdx.x & (kHalf - 1)];
      if (kWarps > 16) s += from[16 + (threadIdx.x & 15)];
#pragma unroll
      for (int d = kHalf / 2; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    return make_float2(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 16));
  }
  __device__ float2 all(float2 v, int turn) {
    add(v, turn);
    ready();
    return get(turn);
  }
};

// A team of kTeam threads holds a row in registers, kPer vectors of kVec elements a
// thread, and loads its next row before it works on this one.
template <class X, class W, bool kRms, int kVec, int kTeam, int kPer, int kTeams>
__global__ void __launch_bounds__(kTeam* kTeams) norm_rows(const NormArgs a) {
  __shared__ float sm[kTeam > 32 ? kTeams * 128 : 1];
  const int team = threadIdx.x / kTeam, at = threadIdx.x % kTeam;
  const int32_t D = static_cast<int32_t>(a.D);
  const X* x = static_cast<const X*>(a.x);
  const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
  const float n = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  typedef Reg<kVec> Row;
  TeamSums<kTeam> sums(sm + team * 128, team);
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
    Row f[kPer];
    typename Row::E s1 = Row::all(0.0f), s2 = s1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        next[i].get(f[i]);
#pragma unroll
        for (int j = 0; j < (kRms ? 0 : Row::kW); ++j) s1 = vadd(s1, f[i].v[j]);
      }
    if (t + step < a.T) load(t + step);
    float m1 = 0.0f;
    if constexpr (!kRms) {
      m1 = sums.all(make_float2(total(s1), 0.0f), turn).x / n;
      turn ^= 1;
      s1 = s2;
    }
    const typename Row::E back = Row::all(-m1);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
#pragma unroll
        for (int j = 0; j < Row::kW; ++j) {
          if (!kRms) {
            f[i].v[j] = vadd(f[i].v[j], back);
            s1 = vadd(s1, f[i].v[j]);
          }
          s2 = vfma(f[i].v[j], f[i].v[j], s2);
        }
      }
    const float2 s = sums.all(make_float2(kRms ? 0.0f : total(s1), total(s2)), turn);
    turn ^= 1;
    const float c = kRms ? 0.0f : s.x / n;
    const float var = s.y / n - c * c;
    const float r = __frsqrt_rn((var < 0.0f ? 0.0f : var) + a.eps);  // (fmaxf would lose a NaN)
    const typename Row::E rs = Row::all(r), cr = Row::all(-c * r);
    X* y = static_cast<X*>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int col = column(i);
      if (col >= D) continue;
      if constexpr (kRms) {
        if (w) {
          Row g;
          load_weight<W, kVec>(w + col, g);
#pragma unroll
          for (int j = 0; j < Row::kW; ++j) f[i].v[j] = vmul(vmul(f[i].v[j], rs), g.v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < Row::kW; ++j) f[i].v[j] = vmul(f[i].v[j], rs);
        }
      } else {
#pragma unroll
        for (int j = 0; j < Row::kW; ++j) f[i].v[j] = vfma(f[i].v[j], rs, cr);
        if (w && b) {
          Row g, h;
          load_weight<W, kVec>(w + col, g);
          load_weight<W, kVec>(b + col, h);
#pragma unroll
          for (int j = 0; j < Row::kW; ++j) f[i].v[j] = vfma(f[i].v[j], g.v[j], h.v[j]);
        } else if (w || b) {
          Row g;
          load_weight<W, kVec>((w ? w : b) + col, g);
#pragma unroll
          for (int j = 0; j < Row::kW; ++j) f[i].v[j] = w ? vmul(f[i].v[j], g.v[j]) : vadd(f[i].v[j], g.v[j]);
        }
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

// A block's sums of dy h and dy, its teams' added up in order, to row blockIdx.x of
// `partial`.  sums: [2][D] of shared memory, where kTeams > 1.
template <bool kRms, int kVec, int kTeam, int kPer, int kTeams>
__device__ __forceinline__ void leave_sums(const NormArgs& a, int team, int at, const Reg<kVec> (&sw)[kPer],
                                           const Reg<kVec>* sb, float* sums) {
  if (!a.partial) return;
  const int32_t D = static_cast<int32_t>(a.D);
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * D;
#pragma unroll 1
  for (int k = 0; k < kTeams; ++k) {
    if (team == k) {
      float* to = k + 1 < kTeams ? sums : out;
      auto leave = [&](const Reg<kVec>& v, int64_t i) {
        if constexpr (kVec == 1) {
          to[i] = k > 0 ? v.v[0] + sums[i] : v.v[0];
        } else if constexpr (kVec == 2) {
          float2 f = unpack2(v.v[0]);
          if (k > 0) f.x += sums[i], f.y += sums[i + 1];
          *reinterpret_cast<float2*>(to + i) = f;  // (D is even)
        } else {
#pragma unroll
          for (int j = 0; j < kVec; j += 4) {  // (D is a multiple of 4)
            const float2 p = unpack2(v.v[j / 2]), q = unpack2(v.v[j / 2 + 1]);
            float4 f = make_float4(p.x, p.y, q.x, q.y);
            if (k > 0) {
              const float4 o = *reinterpret_cast<const float4*>(sums + i + j);
              f = make_float4(f.x + o.x, f.y + o.y, f.z + o.z, f.w + o.w);
            }
            *reinterpret_cast<float4*>(to + i + j) = f;
          }
        }
      };
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int col = (i * kTeam + at) * kVec;
        if (col >= D) continue;
        leave(sw[i], col);
        if constexpr (!kRms) leave(sb[i], D + col);
      }
    }
    if (kTeams > 1) __syncthreads();
  }
}

// The gradients: teams as above.  A thread's columns are the same in every row, so
// that it keeps their sums of dy h and dy in registers, and their weights.
//
// Rows come through a ring in shared memory, of which every thread copies and reads
// its own columns alone: 96 KB of an SM's loads in flight, where a row ahead in
// registers is 32 KB.  A row's sums meet at a barrier while the team is at the first
// half of the next row, and its dx follows, from the ring again: waiting for the sums
// of each row in turn left the SM idle for half of the time (8192 x 8192: 81 us).
__host__ __device__ constexpr int back_slots(int threads, int per = 2) { return threads > 512 || per == 4 ? 3 : 5; }
template <class X, int kVec, int kPer>
constexpr size_t back_ring(int threads) {
  return static_cast<size_t>(back_slots(threads, kPer)) * 2 * kPer * threads * kVec * sizeof(X);
}

template <class X, class W, bool kRms, int kVec, int kTeam, int kPer, int kTeams>
__global__ void __launch_bounds__(kTeam* kTeams, 512 / (kTeam * kTeams) > 0 ? 512 / (kTeam * kTeams) : 1)
    norm_rows_back(const NormArgs a) {
  static_assert(kVec >= 2, "copies of 4 or 16 bytes");
  extern __shared__ __align__(16) uint8_t ring[];  // then the sums, where kTeams > 1
  __shared__ float sm[kTeam > 32 ? kTeams * 128 : 1];
  constexpr int kThreads = kTeam * kTeams, kSlots = back_slots(kThreads, kPer);
  // The weights stay in registers: as they lie in memory where a thread has 32 columns
  // (kPer 4) of 16 bits; a block of 1024 threads has no room for them.
  constexpr bool kRaw = kPer == 4 && sizeof(X) == 2 && sizeof(W) == 2;
  constexpr bool kHold = kThreads <= 512 && !kRaw;
  typedef Reg<kVec> Row;
  typedef typename Row::E E;
  const int team = threadIdx.x / kTeam, at = threadIdx.x % kTeam;
  const int32_t D = static_cast<int32_t>(a.D);
  const X *x = static_cast<const X*>(a.x), *dy = static_cast<const X*>(a.dy);
  const W* w = static_cast<const W*>(a.weight);
  const float n = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  Row sw[kPer], sb[kRms ? 1 : kPer], wv[kHold ? kPer : 1];
  uint4 raw[kRaw ? kPer : 1];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < Row::kW; ++j) sw[i].v[j] = sb[kRms ? 0 : i].v[j] = Row::all(0.0f);
  auto column = [&](int i) { return (i * kTeam + at) * kVec; };
  // Slot s, vector i of x (which = 0) or dy (1) of this thread.
  constexpr uint32_t kBytes = Vec<X, kVec>::kBytes;
  const uint32_t mine = ptx::smem_addr(ring) + threadIdx.x * kBytes;
  auto slot = [&](int s, int which, int i) {
    return mine + static_cast<uint32_t>(((s * 2 + which) * kPer + i) * kThreads) * kBytes;
  };
  auto copy = [&](uint32_t to, const X* from) {
    if constexpr (kBytes == 16)
      ptx::cp_async_16(to, from);
    else
      ptx::cp_async_4(to, from);
  };
  auto fetch = [&](int64_t row, int s) {
    if (row < a.T) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (column(i) < D) {
          copy(slot(s, 0, i), x + row * a.ldx + column(i));
          copy(slot(s, 1, i), dy + row * a.lddy + column(i));
        }
    }
    ptx::cp_async_commit();
  };
  auto stats = [&](int64_t row) {
    if (row >= a.T) return make_float2(0.0f, 0.0f);
    return kRms ? make_float2(0.0f, a.stats[row]) : make_float2(a.stats[2 * row], a.stats[2 * row + 1]);
  };
  auto weights = [&](int i, Row& v) {
    if (w && column(i) < D) {
      load_weight<W, kVec>(w + column(i), v);
    } else {
#pragma unroll
      for (int j = 0; j < Row::kW; ++j) v.v[j] = Row::all(1.0f);
    }
  };
  // x and dy of vector i, from slot s; the weights.
  auto take = [&](int s, int i, Row& f, Row& g, Row& q) {
    Vec<X, kVec> v;
    v.load_shared(slot(s, 0, i));
    v.get(f);
    v.load_shared(slot(s, 1, i));
    v.get(g);
    if constexpr (kHold) {
      q = wv[i];
    } else if constexpr (kRaw) {
      Vec<W, kVec> u;
      u.r = raw[i];
      u.get(q);
    } else {
      weights(i, q);
    }
  };
  // The first half of a row: its sums of q and q h, and its share of the weights'.
  auto first = [&](int s, float2 st) {
    const E back = Row::all(-st.x), rs = Row::all(st.y);
    E s1 = Row::all(0.0f), s2 = s1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        Row h, g, q;
        take(s, i, h, g, q);
#pragma unroll
        for (int j = 0; j < Row::kW; ++j) {
          if (!kRms) h.v[j] = vadd(h.v[j], back);
          h.v[j] = vmul(h.v[j], rs);
          q.v[j] = vmul(g.v[j], q.v[j]);
          sw[i].v[j] = vfma(g.v[j], h.v[j], sw[i].v[j]);
          if (!kRms) {
            sb[kRms ? 0 : i].v[j] = vadd(sb[kRms ? 0 : i].v[j], g.v[j]);
            s1 = vadd(s1, q.v[j]);
          }
          s2 = vfma(q.v[j], h.v[j], s2);
        }
      }
    return make_float2(kRms ? 0.0f : total(s1), total(s2));
  };
  // The second:  dx = r q - h r c2 - r c1.
  auto second = [&](int s, int64_t t, float2 st, float2 sum) {
    const float r = st.y, c1 = kRms ? 0.0f : sum.x / n, c2 = sum.y / n;
    const E back = Row::all(-st.x), rs = Row::all(r), k2 = Row::all(-r * c2), k1 = Row::all(-r * c1);
    X* dx = static_cast<X*>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        Row f, g, q;
        take(s, i, f, g, q);
#pragma unroll
        for (int j = 0; j < Row::kW; ++j) {
          const E h = vmul(kRms ? f.v[j] : vadd(f.v[j], back), rs);
          f.v[j] = vfma(vmul(g.v[j], q.v[j]), rs, kRms ? vmul(h, k2) : vfma(h, k2, k1));
        }
        Vec<X, kVec>::store(dx + column(i), f);
      }
  };
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // Row k of this team is in slot k % kSlots; rows k + 1 .. k + kSlots - 2 are on their
  // way while the team is at row k's first half (and at row k - 1's second).
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) fetch(t0 + s * step, s);
#pragma unroll
  for (int i = 0; i < (kHold ? kPer : 0); ++i) weights(i, wv[i]);
#pragma unroll
  for (int i = 0; i < (kRaw ? kPer : 0); ++i) {
    const uint32_t one = std::is_same<W, __nv_bfloat16>::value ? 0x3f803f80u : 0x3c003c00u;
    raw[i] = make_uint4(one, one, one, one);
    if (w && column(i) < D) raw[i] = *reinterpret_cast<const uint4*>(w + column(i));
  }
  float2 st = stats(t0), last_st = make_float2(0.0f, 0.0f);
  int s = 0, turn = 0;
  TeamSums<kTeam> sums(sm + team * 128, team);
  for (int64_t t = t0; t - step < a.T; t += step, turn ^= 1) {
    const int before = s == 0 ? kSlots - 1 : s - 1;
    const bool again = t > t0;
    const float2 next_st = stats(t + step);  // on its way while this row is worked on
    if (again) sums.ready();
    float2 last = make_float2(0.0f, 0.0f);
    if (kTeam == 32 && again) last = sums.get(0);  // before the next row's take its place
    if (t < a.T) {
      ptx::cp_async_wait<kSlots - 2>();
      sums.add(first(s, st), turn);
    }
    if (kTeam > 32 && again) last = sums.get(turn ^ 1);
    if (again) second(before, t - step, last_st, last);
    fetch(t + (kSlots - 1) * step, before);
    last_st = st;
    st = next_st;
    s = s + 1 == kSlots ? 0 : s + 1;
  }
  ptx::cp_async_wait<0>();
  if (kTeams > 1) __syncthreads();  // the sums take the ring's place
  leave_sums<kRms, kVec, kTeam, kPer, kTeams>(a, team, at, sw, sb, reinterpret_cast<float*>(ring));
}

// The same for rows that are no whole vectors, by elements or pairs of 16-bit ones: a
// row ahead in registers (through the ring, 4 bytes a copy, 2713 x 6563 fp32 took 78 us
// in place of 62).
template <class X, class W, bool kRms, int kVec, int kTeam, int kPer, int kTeams>
__global__ void __launch_bounds__(kTeam* kTeams) norm_rows_back_single(const NormArgs a) {
  extern __shared__ __align__(16) float block_sums_of[];  // [2][D], where kTeams > 1
  __shared__ float sm[kTeam > 32 ? kTeams * 128 : 1];
  typedef Reg<kVec> Row;
  typedef typename Row::E E;
  const int team = threadIdx.x / kTeam, at = threadIdx.x % kTeam;
  const int32_t D = static_cast<int32_t>(a.D);
  const X *x = static_cast<const X*>(a.x), *dy = static_cast<const X*>(a.dy);
  const W* w = static_cast<const W*>(a.weight);
  const float n = static_cast<float>(D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  TeamSums<kTeam> sums(sm + team * 128, team);
  Vec<X, kVec> xn[kPer], gn[kPer];
  float mn = 0.0f, rn = 0.0f;
  Row sw[kPer], sb[kRms ? 1 : kPer], wv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) sw[i].v[0] = sb[kRms ? 0 : i].v[0] = Row::all(0.0f);
  auto column = [&](int i) { return (i * kTeam + at) * kVec; };
  auto fetch = [&](int64_t t) {
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        xn[i].load(x + t * a.ldx + column(i));
        gn[i].load(dy + t * a.lddy + column(i));
      }
    if (!kRms) mn = a.stats[2 * t];
    rn = a.stats[kRms ? t : 2 * t + 1];
  };
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  fetch(t);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    wv[i].v[0] = Row::all(1.0f);
    if (w && column(i) < D) load_weight<W, kVec>(w + column(i), wv[i]);
  }
  for (int turn = 0; t < a.T; t += step, turn ^= 1) {
    const E back = Row::all(-mn), rs = Row::all(rn);
    const float r = rn;
    Row h[kPer], q[kPer], g;
    E s1 = Row::all(0.0f), s2 = s1;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        xn[i].get(h[i]);
        gn[i].get(g);
        h[i].v[0] = vmul(kRms ? h[i].v[0] : vadd(h[i].v[0], back), rs);
        q[i].v[0] = vmul(g.v[0], wv[i].v[0]);
        sw[i].v[0] = vfma(g.v[0], h[i].v[0], sw[i].v[0]);
        if (!kRms) {
          sb[kRms ? 0 : i].v[0] = vadd(sb[kRms ? 0 : i].v[0], g.v[0]);
          s1 = vadd(s1, q[i].v[0]);
        }
        s2 = vfma(q[i].v[0], h[i].v[0], s2);
      }
    fetch(t + step);
    const float2 s = sums.all(make_float2(kRms ? 0.0f : total(s1), total(s2)), turn);
    const E k1 = Row::all(kRms ? 0.0f : -r * (s.x / n)), k2 = Row::all(-r * (s.y / n));
    X* dx = static_cast<X*>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (column(i) < D) {
        q[i].v[0] = vfma(q[i].v[0], rs, kRms ? vmul(h[i].v[0], k2) : vfma(h[i].v[0], k2, k1));
        Vec<X, kVec>::store(dx + column(i), q[i]);
      }
  }
  leave_sums<kRms, kVec, kTeam, kPer, kTeams>(a, team, at, sw, sb, block_sums_of);
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

// The sums of all chunks: 32 columns by kGroups groups of chunks, each in order, then the
// groups in order.  grid (columns / 32, weight or bias).
template <class W, int kGroups>
__global__ void __launch_bounds__(32 * kGroups) norm_dw_sum(const NormArgs a) {
  __shared__ float sm[kGroups][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  W* out = static_cast<W*>(blockIdx.y == 0 ? a.dweight : a.dbias);
  if (!out) return;
  float s = 0.0f;
  if (col < a.D) {
#pragma unroll 8
    for (int64_t c = group; c < a.chunks; c += kGroups) s += a.partial[(2 * c + blockIdx.y) * a.D + col];
  }
  sm[group][lane] = s;
  __syncthreads();
  if (group == 0 && col < a.D) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) s += sm[i][lane];
    narrow(s, out + col);
  }
}

}  // namespace ops
}  // namespace gb300
