// The norms before and after a block, fused with the block's gate, its residual
// scale and the residual sum, forward and backward.
//
//     n = y / rms(y) . w_post        (no w_post: n = y)
//     r = x + scale . gate . n       (no gate: 1)
//     h = r / rms(r) . w_pre         rms(v) = sqrt(mean(v^2) + eps)
//
// One pass reads x and y and writes r and h: 8 bytes an element in bf16 (7 with
// h as INT8 codes), against 14 for the steps one by one.  HBM-bound.  A row
// belongs to one thread block, which holds it in registers between the two
// row sums; h is taken from the unrounded r.
#include <type_traits>

#include "wq_act_fn.cuh"
#include "wq_ff.cuh"
#include "wq_internal.cuh"

namespace wq {
namespace {

// Two fp32 values in one 64-bit register, with the packed arithmetic of sm_100 (one
// instruction for both; each rounded as by itself).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 floats(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// eight bf16 values of a 16-byte vector as four pairs, and back (one rounding)
__device__ __forceinline__ F2 pair_of(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const uint4& v, F2 (&f)[4]) {
  f[0] = pair_of(v.x);
  f[1] = pair_of(v.y);
  f[2] = pair_of(v.z);
  f[3] = pair_of(v.w);
}
__device__ __forceinline__ uint32_t bf16_pair(F2 a) {
  const float2 f = floats(a);
  return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ uint4 pack(const F2 (&f)[4]) {
  return make_uint4(bf16_pair(f[0]), bf16_pair(f[1]), bf16_pair(f[2]), bf16_pair(f[3]));
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

// N sums over the block, to every thread, with one barrier: over each warp, then every
// warp adds the warps' parts, one a lane.  Two buffers alternate from call to call: a
// buffer is written again only after the barrier of the call in between, which every
// reader of it has reached.
template <typename T, int N>
struct BlockSum {
  T (*buf)[N][32];  // [2]
  int turn;
  __device__ void add(T (&v)[N]) {
    const int warps = (int)(blockDim.x >> 5), lane = (int)(threadIdx.x & 31);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (warps == 1) return;
    T(*b)[32] = buf[turn];
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) b[i][threadIdx.x >> 5] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? b[i][lane] : (T)0;
    // (every lane gets the sum, in the same order: lanes past the power of two above
    // `warps` hold zeros)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < 2 * warps)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
  }
};

// The largest bit pattern over a warp, and a sum with it over the block.  Magnitudes
// of fp64 values order as their bits do, with infinities and NaN on top.
__device__ __forceinline__ unsigned long long warp_top(unsigned long long v) {
  const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(v >> 32));
  const unsigned lo = __reduce_max_sync(0xffffffffu, (unsigned)(v >> 32) == hi ? (unsigned)v : 0u);
  return (unsigned long long)hi << 32 | lo;
}

// 1 / sqrt(v) in fp64 to a few units in the last place: two Newton steps
// y <- y (3 - v y^2) / 2 from fp32's (2^-22 -> 2^-43 -> 2^-86).  The correctly rounded
// quotient and root cost every thread of a row some 200 instructions more.
__device__ __forceinline__ double rsqrt_f64(double v) {
  if (!(v > 1e-30 && v < 1e30)) return 1.0 / sqrt(v);
  double y = (double)rsqrtf((float)v);
  const double h = 0.5 * v;
  y = y * fma(-h, y * y, 1.5);
  return y * fma(-h, y * y, 1.5);
}

// 1 / s in fp64, the same way
__device__ __forceinline__ double rcp_f64(float s) {
  if (!(s > 1e-30f && s < 1e30f)) return 1.0 / (double)s;
  double y = (double)(1.f / s);
  const double d = (double)s;
  y = fma(fma(-d, y, 1.0), y, y);
  return fma(fma(-d, y, 1.0), y, y);
}

// Whether each of eight bf16 values is zero or of a magnitude in [2^-E, 2^E], on the bit
// patterns without their signs, two at a time: the least of (pattern - 1), where a zero
// wraps to the top, and the largest pattern.  (An infinity or NaN is past every 2^E.)
template <int E>
__device__ __forceinline__ bool moderate(const uint4& v) {
  constexpr unsigned lo = ((127 - E) << 7) - 1, hi = (127 + E) << 7;
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
  unsigned least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned t = w[i] & 0x7FFF7FFFu;
    least = __viaddmin_u16x2(t, 0xFFFFFFFFu, least);
    most = __vmaxu2(most, t);
  }
  return __vminu2(least, lo << 16 | lo) == (lo << 16 | lo) &&
         __vmaxu2(most, hi << 16 | hi) == (hi << 16 | hi);
}

// Four integers as bytes, each held to -128 .. 127.
__device__ __forceinline__ uint32_t pack_s8(int a, int b, int c, int d) {
  uint32_t hi, r;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(d), "r"(c), "r"(0));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(b), "r"(a), "r"(hi));
  return r;
}

// (volatile: read again in every row, not kept in registers)
__device__ __forceinline__ uint4 ld_again(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

struct NormDev {
  const uint4 *x, *y, *gate, *wpost, *wpre;
  int64_t M, D8, per;
  double scale, eps;
  int stages;  // ring slots
  uint4 *r, *h;
  uint2* hq;
  float *hs, *rpost, *rpre;
};

__device__ __forceinline__ uint4 bf16_ones() {
  return make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
}

// Consecutive rows of N tensors copied ahead into a ring of shared memory, [stages][N]
// [D8] vectors.  Every thread copies (cp.async) and reads only its own vectors, so
// no barrier is needed.  A null tensor's place is left unread.
template <int N, int VPT, bool FULL>
struct RowRing {
  uint4* ring;
  int nv, stages;
  int64_t ahead, end, D8;
  int fill = 0, now = 0;
  __device__ void fetch(const uint4* (&from)[N]) {
    if (ahead < end) {
      uint4* st = ring + fill * N * nv;
      const int64_t at = ahead * D8;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (FULL || v < nv)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (from[i]) cp_async16(st + i * nv + v, from[i] + at + v);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++ahead;
    if (++fill == stages) fill = 0;
  }
  __device__ void begin(const uint4* (&from)[N]) {
    for (int i = 0; i < stages - 1; ++i) fetch(from);
  }
  // asks for a further row (into the slot of the row before, which this thread has
  // read) and returns the next one
  __device__ const uint4* next(const uint4* (&from)[N]) {
    fetch(from);
    if (stages == 4)
      asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 3)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    const uint4* st = ring + now * N * nv;
    if (++now == stages) now = 0;
    return st;
  }
};

// A block takes consecutive rows, VPT 16-byte vectors of each a thread, with the rows
// ahead on their way (one row per block with plain loads left the memory idle during the
// two row sums: 8192 x 8192 took 113 us, this one 104, 5.2 TB/s: two barriers a row with
// 16 warps an SM).  scale gate w_post and w_pre stay in registers.
//
// Sums of squares are fp32, per thread and then over the block.  Squares of values past
// 1.8e19 (or a row of values below 1e-15) leave the range where that holds; such a row
// is summed again in fp64.
//
// EACH: a gate row a token, copied ahead like x and y.
template <int VPT, int MAXT, bool FULL, bool EACH>
__global__ void __launch_bounds__(MAXT, VPT == 4 ? 1 : 2) residual_norm_kernel(const NormDev p) {
  constexpr int NT = EACH ? 3 : 2;
  extern __shared__ uint4 ring[];  // [stages][NT][D8]: x, y, gate
  __shared__ __align__(16) float red[2][1][32];
  __shared__ __align__(16) double wide[2][1][32];
  BlockSum<float, 1> block{red, 0};
  const int nv = (int)p.D8, B = (int)blockDim.x;
  const float inv = 1.f / (8.f * (float)p.D8), eps = (float)p.eps;
  const int64_t m0 = blockIdx.x * p.M / gridDim.x, m1 = (blockIdx.x + 1LL) * p.M / gridDim.x;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();
  grid_launch_dependents();
  RowRing<NT, VPT, FULL> rows{ring, nv, p.stages, m0, m1, p.D8};
  const uint4* from[NT];
  from[0] = p.x;
  from[1] = p.y;
  if constexpr (EACH) from[2] = p.gate;
  rows.begin(from);
  uint4 wn[VPT];
  F2 kk[VPT][4];  // scale gate w_post
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = threadIdx.x + k * B;
    wn[k] = p.wpre && (FULL || v < nv) ? __ldg(p.wpre + v) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[k][j] = f2(0.f);
  }
  int64_t gr = p.gate ? m0 / p.per : 0;
  int64_t gend = m0;  // the first row past the gate row at hand
  for (int64_t m = m0; m < m1; ++m) {
    const uint4* st = rows.next(from);
    if (EACH || m == gend) {
      gend = p.gate ? (gr + 1) * p.per : m1;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        if (FULL || v < nv) {
          F2 w[4];
          unpack(EACH ? st[(NT - 1) * nv + v] : p.gate ? __ldg(p.gate + gr * p.D8 + v) : bf16_ones(), kk[k]);
          unpack(p.wpost ? __ldg(p.wpost + v) : bf16_ones(), w);
#pragma unroll
          for (int j = 0; j < 4; ++j) kk[k][j] = kk[k][j] * (w[j] * f2((float)p.scale));
        }
      }
      ++gr;
    }
    const int64_t at = m * p.D8;
    F2 t[VPT][4];
    // 1 / rms of the values in t, whose squares' sum over this thread is s
    auto inv_rms = [&](F2 s) -> float {
      const float2 h = floats(s);
      float total[1] = {h.x + h.y};
      block.add(total);
      if (total[0] > 1e-30f && total[0] < 1e38f)  // the same for every thread of the block
        return rsqrtf(total[0] * inv + eps);
      double d[1] = {0.0};
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!FULL && (int)threadIdx.x + k * B >= nv) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = floats(t[k][j]);
          d[0] += (double)e.x * (double)e.x + (double)e.y * (double)e.y;
        }
      }
      BlockSum<double, 1>{wide, 0}.add(d);
      __syncthreads();  // its buffer is read
      return (float)(1.0 / sqrt(d[0] / (8.0 * (double)p.D8) + p.eps));
    };
    if (p.y) {
      F2 post = f2(1.f);
      if (p.wpost) {
        F2 s = f2(0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int v = threadIdx.x + k * B;
          if (!FULL && v >= nv) continue;
          unpack(st[nv + v], t[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) s = fma2(t[k][j], t[k][j], s);
        }
        const float rp = inv_rms(s);
        if (threadIdx.x == 0 && p.rpost) p.rpost[m] = rp;
        post = f2(rp);
      }
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        if (!FULL && v >= nv) continue;
        F2 x[4];
        if (!p.wpost) unpack(st[nv + v], t[k]);
        unpack(st[v], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) t[k][j] = fma2(t[k][j] * post, kk[k][j], x[j]);
        p.r[at + v] = pack(t[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        if (!FULL && v >= nv) continue;
        unpack(st[v], t[k]);
      }
    }
    if (!p.wpre) continue;
    F2 s = f2(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!FULL && (int)threadIdx.x + k * B >= nv) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fma2(t[k][j], t[k][j], s);
    }
    const float rn = inv_rms(s);
    if (threadIdx.x == 0 && p.rpre) p.rpre[m] = rn;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * B;
      if (!FULL && v >= nv) continue;
      F2 w[4];
      unpack(wn[k], w);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = w[j] * (t[k][j] * f2(rn));
      p.h[at + v] = pack(w);
    }
  }
}

// h as INT8 codes: rounding to codes has borders, so everything up to the code is fp64
// and the codes are the definition's.  What fp64 costs is conversions (F2F runs at an
// eighth of fp32's rate): gate and w_post are joined in fp32, where their product is
// exact, and so is its product with y (8 + 8 + 8 bits), so one conversion serves the
// three.  That holds while no product leaves fp32's normal range: where a thread's gate and
// w_post are in 2^-40 .. 2^40 and its y in 2^-46 .. 2^46, or zero; a thread with others
// multiplies in fp64 (the test costs 2 to 6%; to redo the row, told by its maximum, cost 11
// to 28%, by the registers that it held).  r w_pre is kept: its largest magnitude gives the
// scale, found beside the sum of squares with one barrier, and one fused multiply-add with
// 1.5 x 2^52 rounds (r w_pre) (1 / (rms s)) to the nearest integer, half to even.  w_pre is
// read in every row, out of L1 (kept in registers it made others spill: 4096 x 4096 47 us,
// so 41).  8192 x 8192 153 us, 3.1 TB/s: conversions and issue slots are at 51% each, with
// 16 warps an SM to hide a row's chain of sums behind.
template <int VPT, int MAXT, bool FULL, bool EACH>
__global__ void __launch_bounds__(MAXT, 1) residual_norm_int8_kernel(const NormDev p) {
  constexpr int NT = EACH ? 3 : 2;
  extern __shared__ uint4 ring[];  // [stages][NT][D8]: x, y, gate
  __shared__ double red[2][1][32];
  __shared__ unsigned long long tops[2][32];
  BlockSum<double, 1> block{red, 0};
  const int nv = (int)p.D8, B = (int)blockDim.x;
  const double inv = 1.0 / (8.0 * (double)p.D8);
  const int64_t m0 = blockIdx.x * p.M / gridDim.x, m1 = (blockIdx.x + 1LL) * p.M / gridDim.x;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();
  grid_launch_dependents();
  RowRing<NT, VPT, FULL> rows{ring, nv, p.stages, m0, m1, p.D8};
  const uint4* from[NT];
  from[0] = p.x;
  from[1] = p.y;
  if constexpr (EACH) from[2] = p.gate;
  rows.begin(from);
  F2 kk[VPT][4];  // gate w_post
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[k][j] = f2(0.f);
  }
  int64_t gr = p.gate ? m0 / p.per : 0;
  int64_t gend = m0;
  bool joined = true;  // this thread's gate and w_post may be joined in fp32
  for (int64_t m = m0; m < m1; ++m) {
    const uint4* st = rows.next(from);
    if (EACH || m == gend) {
      gend = p.gate ? (gr + 1) * p.per : m1;
      joined = true;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        if (FULL || v < nv) {
          const uint4 gv = EACH ? st[(NT - 1) * nv + v] : p.gate ? __ldg(p.gate + gr * p.D8 + v) : bf16_ones();
          const uint4 pv = p.wpost ? __ldg(p.wpost + v) : bf16_ones();
          joined = joined && moderate<40>(gv) && moderate<40>(pv);
          F2 w[4];
          unpack(gv, kk[k]);
          unpack(pv, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) kk[k][j] = kk[k][j] * w[j];
        }
      }
      ++gr;
    }
    const int64_t at = m * p.D8;
    double post = p.scale;
    if (p.y && p.wpost) {
      double v2[1] = {0.0};
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        F2 y[4];
        unpack(FULL || v < nv ? st[nv + v] : zero, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = floats(y[j]);
          v2[0] += (double)e.x * (double)e.x;
          v2[0] += (double)e.y * (double)e.y;
        }
      }
      block.add(v2);
      const double rp = rsqrt_f64(v2[0] * inv + p.eps);
      if (threadIdx.x == 0 && p.rpost) p.rpost[m] = (float)rp;
      post *= rp;
    }
    // y gate w_post
    double t[VPT][8];
    bool plain = joined;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * B;
      plain = plain && moderate<46>(p.y && (FULL || v < nv) ? st[nv + v] : zero);
    }
    if (plain) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        F2 y[4];
        unpack(p.y && (FULL || v < nv) ? st[nv + v] : zero, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = floats(y[j] * kk[k][j]);
          t[k][2 * j] = (double)e.x;
          t[k][2 * j + 1] = (double)e.y;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        const bool in = FULL || v < nv;
#pragma unroll
        for (int j = 0; j < 8; ++j) t[k][j] = 1.0;
        auto times = [&](const uint4& by) {
          F2 f[4];
          unpack(by, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 e = floats(f[j]);
            t[k][2 * j] *= (double)e.x;
            t[k][2 * j + 1] *= (double)e.y;
          }
        };
        times(p.y && in ? st[nv + v] : zero);
        if ((EACH || p.gate) && in) times(EACH ? st[(NT - 1) * nv + v] : __ldg(p.gate + (gr - 1) * p.D8 + v));
        if (p.wpost && in) times(__ldg(p.wpost + v));
      }
    }
    double sum[1] = {0.0};
    unsigned long long top = 0;  // bits of the largest |r w_pre|
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * B;
      F2 x[4], w[4];
      unpack(FULL || v < nv ? st[v] : zero, x);
      unpack(FULL || v < nv ? ld_again(p.wpre + v) : zero, w);
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 xe = floats(x[j]), we = floats(w[j]);
        const double r0 = fma(t[k][2 * j], post, (double)xe.x);
        const double r1 = fma(t[k][2 * j + 1], post, (double)xe.y);
        o[j] = pack_bf16((float)r0, (float)r1);
        sum[0] = fma(r0, r0, sum[0]);
        sum[0] = fma(r1, r1, sum[0]);
        t[k][2 * j] = r0 * (double)we.x;
        t[k][2 * j + 1] = r1 * (double)we.y;
        top = max(top, (unsigned long long)__double_as_longlong(fabs(t[k][2 * j])));
        top = max(top, (unsigned long long)__double_as_longlong(fabs(t[k][2 * j + 1])));
      }
      if (p.y && (FULL || v < nv)) p.r[at + v] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    // (the sum's barrier serves the maximum: its two buffers alternate alike)
    top = warp_top(top);
    if ((threadIdx.x & 31) == 0) tops[m & 1][threadIdx.x >> 5] = top;
    block.add(sum);
    if (B > 32) top = warp_top((int)(threadIdx.x & 31) < (B >> 5) ? tops[m & 1][threadIdx.x & 31] : 0ull);
    const double rn = rsqrt_f64(sum[0] * inv + p.eps);
    if (threadIdx.x == 0 && p.rpre) p.rpre[m] = (float)rn;
    // scale amax / 127 in fp64 (the product with 1 / 127 corrected by its remainder is
    // the quotient), rounded once
    const double amax = __longlong_as_double((long long)top) * rn;
    double quot = amax * (1.0 / 127.0);
    quot = fma(fma(-quot, 127.0, amax), 1.0 / 127.0, quot);
    const float sc = __double2float_rn(quot);
    if (threadIdx.x == 0) p.hs[m] = sc;
    const double by = rn * rcp_f64(sc);
    const bool live = sc > 0.f && sc < INFINITY;  // else (underflow, not a number) codes 0
    // a subnormal scale is rounded coarsely: amax / scale may pass 127.5 there (up to 190).
    // The bytes are held to -128 .. 127 anyway, these to -127
    const bool coarse = sc < 1.17549435e-38f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * B;
      if (FULL || v < nv) {
        uint32_t w[2] = {0u, 0u};
        if (live) {
          int q[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = __double2loint(fma(t[k][j], by, 6755399441055744.0));
          w[0] = pack_s8(q[0], q[1], q[2], q[3]);
          w[1] = pack_s8(q[4], q[5], q[6], q[7]);
          if (coarse) {
            w[0] = __vmaxs4(w[0], 0x81818181u);
            w[1] = __vmaxs4(w[1], 0x81818181u);
          }
        }
        p.hq[at + v] = make_uint2(w[0], w[1]);
        if (p.h) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = pack_bf16((float)(t[k][2 * j] * rn), (float)(t[k][2 * j + 1] * rn));
          p.h[at + v] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
}

// Threads of a block (VPT vectors each; one where rows are so few that a row's own
// latency counts), blocks an SM up to `resident` threads, ring slots that fit.
// FULL: every thread has all its vectors, and the row loop no comparisons (8192 x 8192:
// 104 us without it).  Elsewhere the bf16 kernel's warps skip a vector that none of their
// lanes has (2413 x 13672: 77 -> 66 us; the INT8 kernel gains nothing by that).
template <int VPT, bool I8, bool EACH>
cudaError_t launch_rows(NormDev p, int resident, cudaStream_t st) {
  const int64_t nv = p.D8, slot = (EACH ? 48 : 32) * nv;
  const unsigned threads = (unsigned)(((nv + VPT - 1) / VPT + 31) / 32 * 32);
  int64_t n = resident / threads;
  n = n > 32 ? 32 : n < 1 ? 1 : n;
  const int64_t want = n * device_sm_count();
  // rows evenly over the blocks (ceil(M / blocks) each: INT8 4571 x 1240 24.4 -> 26.6 us,
  // bf16 2413 x 13672 67 -> 70, 30000 x 1024 56 -> 55)
  const unsigned grid = (unsigned)(p.M < want ? p.M : want);
  const int64_t most = (p.M + grid - 1) / grid;
  int64_t stages = (233472 / n - 3072) / slot;
  if (stages > 4) stages = 4;
  if (stages > most + 1) stages = most + 1;
  if (stages < 2) stages = 2;
  p.stages = (int)stages;
  const bool full = (int64_t)threads * VPT == nv;
  void (*kernel)(const NormDev);
  if constexpr (I8)
    kernel = full ? residual_norm_int8_kernel<VPT, VPT == 4 ? 512 : 1024, true, EACH>
                  : residual_norm_int8_kernel<VPT, VPT == 4 ? 512 : 1024, false, EACH>;
  else
    kernel = full ? residual_norm_kernel<VPT, 512, true, EACH> : residual_norm_kernel<VPT, 512, false, EACH>;
  const cudaError_t e = ensure_max_dynamic_smem((const void*)kernel, 225 * 1024);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(grid), threads, (size_t)(stages * slot), st, 1, p);
}

template <bool EACH>
cudaError_t launch_norm(const NormDev& p, cudaStream_t st) {
  // one vector a thread while every SM has a row at most, two up to four rows an SM:
  // the row's own latency counts there
  const int64_t nv = p.D8, sms = device_sm_count();
  const bool few = p.M <= sms, some = p.M <= 4 * sms;
  if (p.hq) {
    if (nv <= 1024 && (few || nv < 64)) return launch_rows<1, true, EACH>(p, 1024, st);
    // four where they fill the lanes of every warp.  us with two / four: 8140 x 2048 46.3 /
    // 40.6, 4096 88.5 / 74.6 (a gate row a token 90.2 / 83.9), 6144 141 / 130, 8192 174 / 153,
    // 39000 x 1024 98.6 / 81.9; 10240 124 / 126; lanes idle in 2560 109 / 125, 4608 115 / 121
    if (nv >= 128 && nv <= 1024 && nv % 128 == 0 && !some)
      return launch_rows<4, true, EACH>(p, 512, st);
    return launch_rows<2, true, EACH>(p, 1024, st);
  }
  if (nv <= 512 && (few || nv < 64)) return launch_rows<1, false, EACH>(p, 1024, st);
  if (nv <= 1024 && (some || nv < 256)) return launch_rows<2, false, EACH>(p, 1024, st);
  return launch_rows<4, false, EACH>(p, 512, st);
}

// ---------------------------------------------------------------- backward
// With rhat = r / rms(r), yhat = y / rms(y), a = dh w_pre, k = scale gate w_post:
//     g  = dr + (a - rhat mean(a rhat)) / rms(r)          = dx
//     dy = (k g - yhat mean(k g yhat)) / rms(y)           (no w_post: scale gate g)
//     dgate = sum over the gate row's tokens of scale w_post g yhat
//     dw_post = sum of scale gate g yhat                   dw_pre = sum of dh rhat
// r is not read: it follows in fp32 from x, y and the kept 1 / rms(y), which are
// read anyway.  The second mean is a sum over g, which holds the first:
//     sum(k yhat g) = sum(k yhat (dr + a / rms(r))) - mean(a rhat) / rms(r) sum(k yhat rhat)
// so three sums are taken over the row at once, with one barrier a row.  While the
// gate row stays the same, dgate and dw_post need one sum only, q = sum of g yhat.
//
// HBM-bound: 12 bytes an element (dr, dh, x, y in; dx, dy out).  A block takes
// consecutive rows; each thread owns up to two 16-byte vectors of every row, copies them
// ahead into shared memory (cp.async, only the thread itself reads them, so no
// barrier), and keeps the column sums.  Blocks' sums leave as one partial row each,
// added in block order by a second kernel: results do not depend on timing.  8140 x
// 4096 83 to 86 us, 4.8 to 4.7 TB/s.  Neither DRAM (52 to 55%) nor the issue slots (50%)
// are full: what bounds it is latency, with one 512-thread block an SM.
struct NormBwdDev {
  const uint4 *dr, *dh, *x, *y, *gate, *wpost, *wpre;
  const float *rpost, *rpre;
  int64_t M, D8, per, rows;
  float scale;
  int stages;
  float* part_w;  // [blocks][2][D]: dw_post, dw_pre
  float* part_g;  // [blocks][2][D]: gate rows begun before / ending after the block's rows
  uint4 *dx, *dy, *dgate;
};

constexpr int kBwdVpt = 2;

// PAIR: rows of more than 8192 columns, shared by the two blocks of a cluster, half the
// columns each; the row sums meet in both blocks' shared memory.
// EACH: a gate row a token.  It is copied ahead like the others, its gradient is the
// row's own, and dw_post, whose sum then changes its factor every row, is kept in q.
template <int MAXT, bool FULL, bool PAIR, bool EACH>
__global__ void __launch_bounds__(MAXT, 1) residual_norm_bwd_kernel(const NormBwdDev p) {
  constexpr int VPT = kBwdVpt, NT = EACH ? 5 : 4;
  extern __shared__ uint4 ring[];  // [stages][NT][nv]: x, y, dr, dh, gate; then fp32 [8 nv]: dw_post
  __shared__ __align__(16) float red[2][3][32];
  __shared__ float met[2][2][4];   // [turn][rank][sum]
  BlockSum<float, 3> block{red, 0};
  const int B = (int)blockDim.x, D = (int)p.D8 * 8;
  const int rank = PAIR ? (int)(blockIdx.x & 1) : 0, id = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  // this block's vectors of a row: nv from voff
  const int voff = PAIR && rank ? (int)((p.D8 + 1) / 2) : 0;
  const int nv = PAIR ? (rank ? (int)(p.D8 / 2) : (int)((p.D8 + 1) / 2)) : (int)p.D8;
  F2* s_post = (F2*)(ring + (int64_t)p.stages * NT * nv);  // four pairs a vector (not EACH)
  const float inv_d = 1.f / (float)D;
  const int64_t m0 = id * p.rows, m1 = min(p.M, m0 + p.rows);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // the other block's shared memory may be written once that block runs: the wait for it
  // stands before the row loop (nothing else is ordered by it)
  if constexpr (PAIR) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  grid_dependency_wait();
  grid_launch_dependents();
  RowRing<NT, VPT, FULL> rows{ring, nv, p.stages, m0, m1, p.D8};
  const uint4* from[NT];
  from[0] = p.x + voff;
  from[1] = p.y ? p.y + voff : nullptr;
  from[2] = p.dr ? p.dr + voff : nullptr;
  from[3] = p.dh ? p.dh + voff : nullptr;
  if constexpr (EACH) from[4] = p.gate + voff;
  rows.begin(from);

  uint4 wn[VPT];
  F2 kk[VPT][4], q[VPT][4], s_pre[VPT][4];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = threadIdx.x + k * B;
    wn[k] = p.wpre && (FULL || v < nv) ? __ldg(p.wpre + voff + v) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      kk[k][j] = q[k][j] = s_pre[k][j] = f2(0.f);
      if (!EACH && (FULL || v < nv)) s_post[4 * v + j] = f2(0.f);
    }
  }
  // scale gate and w_post of this thread's columns (read again where they are needed:
  // twice a gate row)
  const uint4* st = nullptr;
  auto gate_post = [&](int64_t gr, int v, F2 (&g)[4], F2 (&w)[4]) {
    unpack(EACH     ? st[(NT - 1) * nv + v]
           : p.gate ? __ldg(p.gate + gr * p.D8 + voff + v)
                    : bf16_ones(),
           g);
    unpack(p.wpost ? __ldg(p.wpost + voff + v) : bf16_ones(), w);
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = g[j] * f2(p.scale);
  };
  float rp_next = p.wpost ? __ldg(p.rpost + m0) : 1.f, rn_next = p.wpre ? __ldg(p.rpre + m0) : 0.f;
  int64_t gr = p.gate ? m0 / p.per : 0;                    // this row's gate row
  int64_t gend = p.gate ? min(m1, (gr + 1) * p.per) : m1;  // the first row past it, here
  bool first = true, fresh = true;
  if constexpr (PAIR) asm volatile("barrier.cluster.wait;" ::: "memory");
  for (int64_t m = m0; m < m1; ++m) {
    const float rp = rp_next, rn = rn_next;
    if (m + 1 < m1) {
      if (p.wpost) rp_next = __ldg(p.rpost + m + 1);
      if (p.wpre) rn_next = __ldg(p.rpre + m + 1);
    }
    st = rows.next(from);
    if (EACH || fresh) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        F2 w[4];
        if (FULL || v < nv) {
          gate_post(gr, v, kk[k], w);
#pragma unroll
          for (int j = 0; j < 4; ++j) kk[k][j] = kk[k][j] * w[j];
        }
      }
      fresh = false;
    }

    F2 t[VPT][4], rh[VPT][4];
    F2 dot = f2(0.f), a1 = f2(0.f), a2 = f2(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * B;
      const bool in = FULL || v < nv;
      F2 f[4], w[4], ky[4];
      unpack(in && p.y ? st[nv + v] : zero, ky);
      unpack(in ? st[v] : zero, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ky[j] = ky[j] * f2(rp) * kk[k][j];  // k yhat (k / rms(y) may leave fp32)
        rh[k][j] = (f[j] + ky[j]) * f2(rn);
      }
      unpack(in && p.dr ? st[2 * nv + v] : zero, t[k]);
      if (p.wpre) {
        unpack(in ? st[3 * nv + v] : zero, f);
        unpack(wn[k], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 a = f[j] * w[j];
          s_pre[k][j] = fma2(f[j], rh[k][j], s_pre[k][j]);
          dot = fma2(a, rh[k][j], dot);
          t[k][j] = fma2(f2(rn), a, t[k][j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a1 = fma2(ky[j], t[k][j], a1);
        a2 = fma2(ky[j], rh[k][j], a2);
      }
    }
    const float2 e0 = floats(dot), e1 = floats(a1), e2 = floats(a2);
    float sums[3] = {e0.x + e0.y, e1.x + e1.y, e2.x + e2.y};
    block.add(sums);
    if constexpr (PAIR) {
      const int turn = (int)(m & 1);
      if (threadIdx.x < 6) {
        // both blocks' sums to both blocks, added in rank order
        const int i = (int)threadIdx.x % 3;
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(&met[turn][rank][i]);
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(threadIdx.x / 3));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(i == 0 ? sums[0] : i == 1 ? sums[1] : sums[2])
                     : "memory");
      }
      asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
#pragma unroll
      for (int i = 0; i < 3; ++i) sums[i] = met[turn][0][i] + met[turn][1][i];
    }
    const float c1 = rn * (sums[0] * inv_d);                           // g = t - rhat c1
    const float c2 = p.wpost ? (sums[1] - c1 * sums[2]) * inv_d : 0.f;  // mean(k g yhat)
    const int64_t at = m * p.D8 + voff;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * B;
      if (FULL || v < nv) {
        F2 yh[4], o[4];
        unpack(p.y ? st[nv + v] : zero, yh);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          yh[j] = yh[j] * f2(rp);
          t[k][j] = fma2(rh[k][j], f2(-c1), t[k][j]);
          o[j] = fma2(yh[j], f2(-c2), kk[k][j] * t[k][j]) * f2(rp);
          if (EACH)
            yh[j] = t[k][j] * yh[j];
          else
            q[k][j] = fma2(t[k][j], yh[j], q[k][j]);
        }
        if constexpr (EACH) {
          F2 w[4], gg[4];
          gate_post(m, v, gg, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            q[k][j] = fma2(gg[j], yh[j], q[k][j]);
            w[j] = w[j] * f2(p.scale) * yh[j];
          }
          if (p.dgate) p.dgate[at + v] = pack(w);
        }
        p.dx[at + v] = pack(t[k]);
        if (p.dy) p.dy[at + v] = pack(o);
      }
    }
    // the last of this block's rows of a gate row: its sums leave
    if (!EACH && m + 1 == gend) {
      const int64_t g0 = gr * p.per, g1 = min(p.M, g0 + p.per);
      const bool whole = g0 >= m0 && g1 <= m1;
      F2* slot = (F2*)(p.part_g + (id * 2LL + (first ? 0 : 1)) * D + 8 * voff);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * B;
        if (FULL || v < nv) {
          F2 w[4], gg[4];
          gate_post(gr, v, gg, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s_post[4 * v + j] = fma2(gg[j], q[k][j], s_post[4 * v + j]);
            w[j] = w[j] * f2(p.scale) * q[k][j];
            q[k][j] = f2(0.f);
          }
          if (p.dgate) {
            if (whole)
              p.dgate[gr * p.D8 + voff + v] = pack(w);
            else
#pragma unroll
              for (int j = 0; j < 4; ++j) slot[4 * v + j] = w[j];
          }
        }
      }
      first = false;
      fresh = true;
      ++gr;
      gend = min(m1, (gr + 1) * p.per);
    }
  }
  F2* part = (F2*)(p.part_w + id * 2LL * D + 8 * voff);
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = threadIdx.x + k * B;
    if (FULL || v < nv)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        part[4 * v + j] = EACH ? q[k][j] : s_post[4 * v + j];
        part[D / 2 + 4 * v + j] = s_pre[k][j];
      }
  }
}

// The blocks' partial column sums: 32 columns a thread block, several threads to a
// column, each a fixed share of the partial rows, then these in order.
// blockIdx.y 0: dw_post, 1: dw_pre, 2 + i: gate rows i, i + (gridDim.y - 2), ...
// that lie in several blocks.
__global__ void __launch_bounds__(1024)
    norm_bwd_reduce_kernel(const float* __restrict__ part_w, const float* __restrict__ part_g,
                           int64_t M, int64_t D, int64_t per, int64_t rows, int64_t ctas,
                           int64_t gates, uint16_t* __restrict__ dwpost,
                           uint16_t* __restrict__ dwpre, uint16_t* __restrict__ dgate) {
  __shared__ float part[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, grps = blockDim.x >> 5;
  const int64_t c = blockIdx.x * 32LL + lane;
  // rows b0, b0 + step, ... up to b1 of a [.., D] array, added over the block
  auto column = [&](const float* at, int64_t n, int64_t stride) -> float {
    float s = 0.f;
    if (c < D)
#pragma unroll 8
      for (int64_t i = grp; i < n; i += grps) s += __ldg(at + i * stride + c);
    __syncthreads();  // the sums of the call before are read
    part[grp][lane] = s;
    __syncthreads();
    s = 0.f;
    if (grp == 0)
      for (int i = 0; i < grps; ++i) s += part[i][lane];
    return s;
  };
  if (blockIdx.y < 2) {
    uint16_t* out = blockIdx.y ? dwpre : dwpost;
    if (!out) return;
    const float s = column(part_w + blockIdx.y * D, ctas, 2 * D);
    if (grp == 0 && c < D) out[c] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    return;
  }
  auto first_part = [&](int64_t g0) -> float {
    // the first block's part lies in its second slot where another gate row comes before
    const int64_t b0 = g0 / rows;
    return c < D ? __ldg(part_g + (b0 * 2 + (g0 > b0 * rows ? 1 : 0)) * D + c) : 0.f;
  };
  if (per / rows < 16) {  // few parts a gate row: a warp of the block takes one by itself
    for (int64_t g = (int64_t)(blockIdx.y - 2) * grps + grp; g < gates; g += (int64_t)(gridDim.y - 2) * grps) {
      const int64_t g0 = g * per, g1 = min(M, g0 + per);
      const int64_t b0 = g0 / rows, b1 = (g1 - 1) / rows;
      if (b0 == b1 || c >= D) continue;  // one block has written it
      float s = first_part(g0);
      for (int64_t b = b0 + 1; b <= b1; ++b) s += __ldg(part_g + b * 2 * D + c);
      dgate[g * D + c] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    }
    return;
  }
  for (int64_t g = blockIdx.y - 2; g < gates; g += gridDim.y - 2) {
    const int64_t g0 = g * per, g1 = min(M, g0 + per);
    const int64_t b0 = g0 / rows, b1 = (g1 - 1) / rows;
    if (b0 == b1) continue;  // one block has written it
    const float head = first_part(g0);
    const float s = head + column(part_g + (b0 + 1) * 2 * D, b1 - b0, 2 * D);
    if (grp == 0 && c < D) dgate[g * D + c] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  }
}

// Threads of a backward block, blocks an SM (512 threads in all, 128 registers each),
// blocks a row, and ring slots that fit its shared memory.
struct BwdShape {
  int threads, per_sm, cluster, stages;
  int64_t nv;  // vectors of a row that a block owns, at most
};
BwdShape bwd_shape(int64_t D, bool each = false) {
  BwdShape b;
  b.cluster = D > 8192 ? 2 : 1;
  b.nv = (D / 8 + b.cluster - 1) / b.cluster;
  b.threads = (int)(((b.nv + kBwdVpt - 1) / kBwdVpt + 31) / 32 * 32);
  b.per_sm = b.threads >= 512 ? 1 : 512 / b.threads;
  const int64_t room = 233472 / b.per_sm - 1024 - 1024 - (each ? 0 : 32) * b.nv;  // reserved; static; dw_post
  const int64_t st = room / ((each ? 80 : 64) * b.nv);
  b.stages = (int)(st > 4 ? 4 : st < 1 ? 1 : st);
  return b;
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs& a) {
  NormDev p;
  p.x = (const uint4*)a.x;
  p.y = (const uint4*)a.y;
  p.gate = (const uint4*)a.gate;
  p.wpost = (const uint4*)a.wpost;
  p.wpre = (const uint4*)a.wpre;
  p.M = a.M;
  p.D8 = a.D / 8;
  p.per = a.per;
  p.scale = a.scale;
  p.eps = a.eps;
  p.r = (uint4*)a.r;
  p.h = (uint4*)a.h;
  p.hq = (uint2*)a.hq;
  p.hs = a.hs;
  p.rpost = a.rpost;
  p.rpre = a.rpre;
  return p.gate && p.per == 1 ? launch_norm<true>(p, a.stream) : launch_norm<false>(p, a.stream);
}

void norm_bwd_grid(int64_t M, int64_t D, int64_t* rows, int64_t* ctas) {
  const BwdShape b = bwd_shape(D);
  const int64_t want = 148 * b.per_sm / b.cluster;
  *rows = M < want ? 1 : (M + want - 1) / want;
  // A block costs three to four fp32 rows of sums, written and read again, as much as two
  // rows of the tensors; a row costs its latency.  Both together are least near
  // sqrt(M / 64) rows a block: 1000 x 1024 27 us with one row, 15.6 with four, 28 with
  // sixteen; 300 x 1024 10.9, 9.4 (two), 27; 3000 x 512 23.4, 21.3 (seven), 28; from
  // twelve rows on more gain nothing (16000 x 256 39.5 with seven, 36.6 with twelve)
  while (*rows < 12 && (2 * *rows + 1) * (2 * *rows + 1) * 16 < M) ++*rows;
  *ctas = (M + *rows - 1) / *rows;
}

cudaError_t launch_residual_norm_bwd(const NormBwdArgs& a) {
  NormBwdDev p;
  p.dr = (const uint4*)a.dr;
  p.dh = (const uint4*)a.dh;
  p.x = (const uint4*)a.x;
  p.y = (const uint4*)a.y;
  p.gate = (const uint4*)a.gate;
  p.wpost = (const uint4*)a.wpost;
  p.wpre = (const uint4*)a.wpre;
  p.rpost = a.rpost;
  p.rpre = a.rpre;
  p.M = a.M;
  p.D8 = a.D / 8;
  p.per = a.gate ? a.per : a.M;
  p.scale = (float)a.scale;
  int64_t ctas;
  norm_bwd_grid(a.M, a.D, &p.rows, &ctas);
  p.part_w = a.partial;
  p.part_g = a.partial + ctas * 2 * a.D;
  p.dx = (uint4*)a.dx;
  p.dy = (uint4*)a.dy;
  p.dgate = (uint4*)a.dgate;
  const bool each = a.gate && a.per == 1;
  const BwdShape b = bwd_shape(a.D, each);
  p.stages = b.stages;
  const size_t smem = (size_t)((b.stages * (each ? 80 : 64) + (each ? 0 : 32)) * b.nv);
  const bool full = (int64_t)b.threads * kBwdVpt * b.cluster == p.D8;
  auto pick = [&](auto pair, auto each) {
    constexpr bool P = decltype(pair)::value, E = decltype(each)::value;
    return full ? residual_norm_bwd_kernel<512, true, P, E> : residual_norm_bwd_kernel<512, false, P, E>;
  };
  const std::true_type yes;
  const std::false_type no;
  auto kernel = b.cluster == 2 ? (each ? pick(yes, yes) : pick(yes, no))
                               : (each ? pick(no, yes) : pick(no, no));
  cudaError_t e = ensure_max_dynamic_smem((const void*)kernel, 226 * 1024);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kernel, dim3((unsigned)(ctas * b.cluster)), (unsigned)b.threads, smem, a.stream,
                       (unsigned)b.cluster, p);
  if (e != cudaSuccess) return e;
  const int64_t gates = a.dgate && a.per > 1 ? (a.M + a.per - 1) / a.per : 0;
  const unsigned reducers = ctas > 1024 ? 1024 : 512;
  int64_t y = a.per / p.rows < 16 ? (gates + reducers / 32 - 1) / (reducers / 32) : gates;
  y = 2 + (y < 1024 ? y : 1024);
  return launch_dependent(norm_bwd_reduce_kernel, dim3((unsigned)((a.D + 31) / 32), (unsigned)y),
                          reducers, 0, a.stream, 1, (const float*)p.part_w, (const float*)p.part_g, a.M,
                          a.D, a.per, p.rows, ctas, gates, (uint16_t*)a.dwpost,
                          (uint16_t*)a.dwpre, (uint16_t*)a.dgate);
}

}  // namespace wq
