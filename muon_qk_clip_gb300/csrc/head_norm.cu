// RMS norm of every query and key head with the rotary embedding in the same
// pass, and its gradient.  Per token t and head h, over the d features of the
// head, with the rotation R of the token's position on the last `rot` of them
// (interleaved pairs, angle position * theta^(-2 k / rot)):
//
//   rstd = 1 / sqrt(mean(x^2) + eps),   y = R (x rstd w)
//   dz = R^T dy,   xhat = x rstd,   g = w dz,
//   dx = rstd (g - xhat mean(g xhat)),   dw = sum over tokens and heads of dz xhat
//
// Queries and keys share one launch: a warp takes a token and a range of its
// query or key heads, and needs the token's sines and cosines once for them.  A
// head's row lies over the fewest lanes that hold it, 16 bytes each (16 lanes for 128
// bf16 features, two heads per warp), or four pairs each where rows are not of whole
// 16 bytes; its sums go over these lanes' shuffles.
//
// Bound by memory: 16384 tokens of 32 / 8 heads of 128 in bf16 56 us, 6.0 TB/s (a copy of
// as much takes 53), gradient 84.5, 5.95; of 256 in fp32 6.3 and 6.0.  Rows of pairs are
// bound by issue: 8192 tokens of 32 / 8 heads of width 90 in bf16 38.5 us, 3.1 TB/s (of
// two-byte accesses without copies ahead 133), in fp32 46.5, 5.1.
//
// Turns: a pair's frequency in turns per position is kept as a 64-bit fraction
// of a turn (from fp64 on the host), and its product with the position, taken
// modulo 2^64, is the turn at the position: exact for every 32-bit position
// (negative ones too) but for the frequency's own rounding, a few 2^-53 of it.
// Its top 32 bits become an fp32 number of half turns for sincospif.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/muonclip.h"
#include "common.cuh"
#include "fastdiv.cuh"
#include "kernels.h"

namespace mc {
namespace {
namespace hn {

// The forward's blocks are small: each leaves its places to the next as its warps end.
// (16384 tokens, 32 / 8 heads of 128, bf16: eight blocks of 128 threads per SM take 56
// us, six 61, nine with spills 60; four of 256 60, three 65; 64 threads 71 and more.
// The gradient, whose blocks stay: two of 256 84.5 us, four of 128 85.)
constexpr int kFrontThreads = 128, kFrontWarps = kFrontThreads / 32;
constexpr int kThreads = 256, kWarps = kThreads / 32;        // of the gradient
constexpr int kMaxPairs = MC_HEAD_MAX / 2;
constexpr int kFlight = 2;                        // rows of a lane per step of the loop
// Blocks that an SM holds at once; of the gradient, and blocks (rows of weight sums)
// at most: one wave.  (Gradient of 8192 tokens, 32 / 8 heads, two blocks and one: bf16
// of width 90 65 us and 78, fp32 of 90 84 and 83, of 192, two 16-byte parts a lane, 133
// and 125.)
__host__ __device__ constexpr int front_blocks(int nu) { return nu == 1 ? 8 : nu == 2 ? 7 : 6; }
__host__ __device__ constexpr int back_blocks(int nu) { return nu == 2 ? 1 : 2; }
constexpr int kBackGrid = 152 * 2;

struct Side {                                     // queries or keys
  const void* x;                                  // the norm's input
  const void* dy;                                 // gradient only
  void* out;                                      // y, or dx
  const void* w;
  long long xt, xh, gt, gh, ot, oh;               // strides: token, head
  int heads;
};
struct Params {
  Side side[2];
  unsigned long long turn[kMaxPairs];             // of pair k, in 2^-64 turns per position
  const int* positions;                           // or null: the token's number
  float* rstd;                                    // [T, heads of both]; null without a norm
  float* part;                                    // gradient: [blocks][2][d] weight sums, or null
  int T, d, rot, heads;
  int lanes;                                      // per row: a power of two
  int span;                                       // heads per unit of work, whole steps of a warp's loop
  int pieces[2];                                  // units per token and side
  float eps, inv_d;
  FastDiv div_pieces[3];                          // by the units of a token: of queries, of keys, of both
};

using Two = unsigned long long;                   // two fp32
// V neighbouring features of a row, in registers as they lie in memory.
template <typename T, int V>
struct Feat;
template <>
struct Feat<__nv_bfloat16, 8> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void fill(uint32_t x) { w = make_uint4(x, x, x, x); }
  __device__ void zero() { fill(0u); }
  __device__ void ones() { fill(0x3f803f80u); }
  __device__ void get(Two (&x)[4]) const {
    const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = two(__uint_as_float(e[i] << 16), __uint_as_float(e[i] & 0xffff0000u));
  }
  __device__ static void store(__nv_bfloat16* p, const Two (&x)[4]) {
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      untwo(x[i], a, b);
      const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
      e[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(e[0], e[1], e[2], e[3]);
  }
};
template <>
struct Feat<float, 4> {
  float4 w;
  __device__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ void fill(float x) { w = make_float4(x, x, x, x); }
  __device__ void zero() { fill(0.f); }
  __device__ void ones() { fill(1.f); }
  __device__ void get(Two (&x)[2]) const { x[0] = two(w.x, w.y); x[1] = two(w.z, w.w); }
  __device__ static void store(float* p, const Two (&x)[2]) {
    float4 w;
    untwo(x[0], w.x, w.y);
    untwo(x[1], w.z, w.w);
    *reinterpret_cast<float4*>(p) = w;
  }
};
template <typename T>
struct Feat<T, 2> {                               // a pair, whatever its alignment
  float a, b;
  __device__ static float in(float v) { return v; }
  __device__ static float in(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static void to(float* p, float v) { *p = v; }
  __device__ static void to(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  __device__ void load(const T* p) { a = in(p[0]); b = in(p[1]); }
  __device__ void load_whole(const void* p) {     // aligned to its size
    if constexpr (sizeof(T) == 4) {
      const float2 w = *static_cast<const float2*>(p);
      a = w.x;
      b = w.y;
    } else {
      const uint32_t w = *static_cast<const uint32_t*>(p);
      a = __uint_as_float(w << 16);
      b = __uint_as_float(w & 0xffff0000u);
    }
  }
  __device__ void zero() { a = b = 0.f; }
  __device__ void ones() { a = b = 1.f; }
  __device__ void get(Two (&x)[1]) const { x[0] = two(a, b); }
  __device__ static void store(T* p, const Two (&x)[1]) {
    float a, b;
    untwo(x[0], a, b);
    to(p, a);
    to(p + 1, b);
  }
  __device__ static void store_whole(T* p, const Two (&x)[1]) {
    float2 w;
    untwo(x[0], w.x, w.y);
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2*>(p) = w;
    } else {
      const __nv_bfloat162 r = __floats2bfloat162_rn(w.x, w.y);
      *reinterpret_cast<__nv_bfloat162*>(p) = r;
    }
  }
};

// A lane's features are V from column V * (its lane of the row + lanes * u), u <
// NU, as long as they are below d.  Sine and cosine per pair; those below the
// rotated part turn by nothing.
template <int V, int NU, bool FAST>
struct Turn {
  float c[NU][V / 2], s[NU][V / 2];
  __device__ void at(const Params& p, int pos, int sub) {
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const int col = V * (sub + p.lanes * u) + 2 * k, pair = (col - (p.d - p.rot)) / 2;
        c[u][k] = 1.f;
        s[u][k] = 0.f;
        if (col < p.d && col >= p.d - p.rot) {
          const long long turn = (long long)(p.turn[pair] * (unsigned long long)(long long)pos);
          const float half = (float)(int)(turn >> 32) * 0x1p-31f;             // of a turn, within +-1
          // bf16 rounds to 2^-9: the hardware's sine and cosine, good to 2^-21 absolute
          // within +-pi, do; fp32 takes the exact ones
          if (FAST) __sincosf(half * 3.14159265358979f, &s[u][k], &c[u][k]);
          else sincospif(half, &s[u][k], &c[u][k]);
        }
      }
  }
};
// Sums over the lanes of a row, of N rows at once (a chain of shuffles has their
// latency: several rows' chains side by side).
template <int N>
__device__ inline void row_sums(float (&v)[N], int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
}

// A lane's weights of one side.
template <typename T, int V, int NU>
__device__ inline void load_weight(const Params& p, const void* w, int sub, Two (&x)[NU][V / 2]) {
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int col = V * (sub + p.lanes * u);
    Feat<T, V> f;
    f.ones();
    if (w && col < p.d) f.load(static_cast<const T*>(w) + col);
    f.get(x[u]);
  }
}
__device__ inline float both(Two v) {
  float a, b;
  untwo(v, a, b);
  return a + b;
}

// A thread's rows on their way: their parts are copied asynchronously to places in
// shared memory that only this thread reads, kDepth steps of F rows ahead, so that
// loads in flight take no registers.  (With two steps of them in registers the
// gradient took 103 us instead of 84.5 for 16384 tokens of 32 / 8 heads of 128.)  Parts
// are 16 bytes, or pairs where rows are aligned to those only (WHOLE); pairs of any
// alignment are loaded where they are used.
constexpr int kDepth = 3;
template <int BYTES>
__device__ inline void copy_part(void* to, const void* from, bool there) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(to)), "l"(from), "n"(BYTES), "r"(there ? BYTES : 0) : "memory");
}
__device__ inline void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ inline void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, int V, int NU, bool WHOLE, int F, int THREADS>
struct Rows {
  static constexpr int kPart = V * (int)sizeof(T);
  char* fifo;                                     // this thread's first place
  const T* base;                                  // the lane's first column of its first row (there if left and cols are positive)
  const T* any;                                   // an address of the operand, for copies of nothing
  long long pitch;                                // of rows that this lane meets in turn
  int left;                                       // rows that it meets
  int cols;                                       // columns from base's to the row's end
  int lanes;
  __device__ char* place(int step, int n, int u) const { return fifo + (((step % kDepth) * F + n) * NU + u) * THREADS * kPart; }
  __device__ void issue(int step) {
    if constexpr (WHOLE) {
#pragma unroll
      for (int n = 0; n < F; ++n)
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int i = step * F + n, col = V * lanes * u;
          const bool there = i < left && col < cols;
          copy_part<kPart>(place(step, n, u), there ? base + i * pitch + col : any, there);
        }
    }
  }
  __device__ void get(int step, int n, int u, Two (&x)[V / 2]) const {
    Feat<T, V> f;
    if constexpr (WHOLE) {
      if constexpr (V == 2) f.load_whole(place(step, n, u));
      else f.load(reinterpret_cast<const T*>(place(step, n, u)));
    } else {
      const int i = step * F + n, col = V * lanes * u;
      f.zero();
      if (i < left && col < cols) f.load(base + i * pitch + col);
    }
    f.get(x);
  }
  __device__ static void put(T* p, const Two (&x)[V / 2]) {
    if constexpr (V == 2 && WHOLE) Feat<T, V>::store_whole(p, x);
    else Feat<T, V>::store(p, x);
  }
};

// NORM: false for heads that are rotated (and weighted) only.  A kernel of its own: the choice at
// run time took a hundredth of the gradient's time.
template <typename T, int V, int NU, bool WHOLE, bool NORM>
__global__ void __launch_bounds__(kFrontThreads, front_blocks(NU)) head_norm_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) char fifo[];
  await_previous();
  release_next();
  const int lane = threadIdx.x & 31, sub = lane & (p.lanes - 1), rows = 32 / p.lanes, group = lane / p.lanes;
  const long long unit = (long long)blockIdx.x * kFrontWarps + (threadIdx.x >> 5);
  const int pieces = p.pieces[0] + p.pieces[1];
  if (unit >= (long long)p.T * pieces) return;
  const int t = (int)fastdiv((uint32_t)unit, p.div_pieces[2]), r = (int)unit - t * pieces, side = r >= p.pieces[0];
  const Side& S = p.side[side];
  const int from = (r - side * p.pieces[0]) * p.span, to = min(S.heads, from + p.span), base = side ? p.side[0].heads : 0;
  const int steps = (to - from + kFlight * rows - 1) / (kFlight * rows);
  using R = Rows<T, V, NU, WHOLE, kFlight, kFrontThreads>;
  R x;
  x.fifo = fifo + threadIdx.x * R::kPart;
  x.any = static_cast<const T*>(S.x);
  x.base = x.any + t * S.xt + (from + group) * S.xh + V * sub;
  x.pitch = rows * S.xh;
  x.left = (to - from - group + rows - 1) / rows;
  x.cols = p.d - V * sub;
  x.lanes = p.lanes;
  T* y = static_cast<T*>(S.out) + t * S.ot + (from + group) * S.oh + V * sub;
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    if (i < steps) x.issue(i);
    copies_end();
  }
  // the weight goes into the rotation: (a, b) -> (a w0 c - b w1 s, a w0 s + b w1 c)
  float ac[NU][V / 2], bs[NU][V / 2], as[NU][V / 2], bc[NU][V / 2];
  {
    Two w[NU][V / 2];
    load_weight<T, V, NU>(p, S.w, sub, w);
    Turn<V, NU, sizeof(T) == 2> turn;
    turn.at(p, p.positions ? p.positions[t] : t, sub);
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        float w0, w1;
        untwo(w[u][k], w0, w1);
        ac[u][k] = w0 * turn.c[u][k];
        as[u][k] = w0 * turn.s[u][k];
        bc[u][k] = w1 * turn.c[u][k];
        bs[u][k] = w1 * turn.s[u][k];
      }
  }
  float* rstds = p.rstd + (long long)t * p.heads + base + from + group;
  for (int i = 0; i < steps; ++i) {
    copies_wait<kDepth - 1>();
    float sums[kFlight];
#pragma unroll
    for (int n = 0; n < kFlight; ++n) {
      Two sum = 0;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        Two v[V / 2];
        x.get(i, n, u, v);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) sum = fma2(v[k], v[k], sum);
      }
      sums[n] = both(sum);
    }
    row_sums(sums, p.lanes);
#pragma unroll
    for (int n = 0; n < kFlight; ++n) {
      const int h = i * kFlight + n;               // of this lane's rows
      if (h >= x.left) continue;
      const float rstd = NORM ? rsqrtf(fmaf(sums[n], p.inv_d, p.eps)) : 1.f;
      if (NORM && sub == 0) rstds[h * rows] = rstd;
      const Two r2 = two(rstd, rstd);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        Two v[V / 2];
        x.get(i, n, u, v);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          float a, b;
          untwo(mul2(v[k], r2), a, b);
          v[k] = two(fmaf(-b, bs[u][k], a * ac[u][k]), fmaf(b, bc[u][k], a * as[u][k]));
        }
        if (V * p.lanes * u < x.cols) R::put(y + h * (rows * S.oh) + V * p.lanes * u, v);
      }
    }
    if (i + kDepth < steps) x.issue(i + kDepth);
    copies_end();
  }
}

template <typename T, int V, int NU, bool WHOLE, bool NORM>
__global__ void __launch_bounds__(kThreads, back_blocks(NU)) head_norm_back_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) char fifo[];    // rows on their way; then [2][rows of all warps][d] weight sums
  await_previous();
  release_next();
  const int lane = threadIdx.x & 31, sub = lane & (p.lanes - 1), rows = 32 / p.lanes, group = lane / p.lanes;
  const int warps = (int)gridDim.x * kWarps, all = kWarps * rows;
  constexpr int F = kFlight;
  using R = Rows<T, V, NU, WHOLE, F, kThreads>;
  float* sums = reinterpret_cast<float*>(fifo + (WHOLE ? 2 * kDepth * F * NU * kThreads * R::kPart : 0));
  // queries, then keys: one side's weight and its sums at a time in registers
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const Side& S = p.side[side];
    const int base = side ? p.side[0].heads : 0, pieces = p.pieces[side];
    Two w[NU][V / 2], dw[NU][V / 2];               // (no keys: no weight either, and sums of nothing)
    load_weight<T, V, NU>(p, S.w, sub, w);
#pragma unroll
    for (int i = 0; i < NU * V / 2; ++i) dw[i / (V / 2)][i % (V / 2)] = 0;
    const long long units = (long long)p.T * pieces;
    for (long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); unit < units; unit += warps) {
      const int t = (int)fastdiv((uint32_t)unit, p.div_pieces[side]);
      const int from = ((int)unit - t * pieces) * p.span, to = min(S.heads, from + p.span);
      const int steps = (to - from + F * rows - 1) / (F * rows);
      R x, g;
      x.fifo = fifo + threadIdx.x * R::kPart;
      g.fifo = x.fifo + kDepth * F * NU * kThreads * R::kPart;
      x.any = static_cast<const T*>(S.x);
      g.any = static_cast<const T*>(S.dy);
      x.base = x.any + t * S.xt + (from + group) * S.xh + V * sub;
      g.base = g.any + t * S.gt + (from + group) * S.gh + V * sub;
      x.pitch = rows * S.xh;
      g.pitch = rows * S.gh;
      x.left = g.left = (to - from - group + rows - 1) / rows;
      x.cols = g.cols = p.d - V * sub;
      x.lanes = g.lanes = p.lanes;
      T* o = static_cast<T*>(S.out) + t * S.ot + (from + group) * S.oh + V * sub;
      const float* rs = p.rstd + (long long)t * p.heads + base + from + group;
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        if (i < steps) {
          x.issue(i);
          g.issue(i);
        }
        copies_end();
      }
      float r[F], r1[F];                          // rstd of this step's rows, and of the next one's
      auto load_r = [&](int i) {
#pragma unroll
        for (int n = 0; n < F; ++n) r1[n] = !NORM ? 1.f : i * F + n < x.left ? rs[(i * F + n) * rows] : 0.f;
      };
      load_r(0);
      Turn<V, NU, sizeof(T) == 2> turn;
      turn.at(p, p.positions ? p.positions[t] : t, sub);
      for (int i = 0; i < steps; ++i) {
#pragma unroll
        for (int n = 0; n < F; ++n) r[n] = r1[n];
        load_r(i + 1);
        copies_wait<kDepth - 1>();
        Two a[F][NU][V / 2], b[F][NU][V / 2];
        float dots[F];
#pragma unroll
        for (int n = 0; n < F; ++n) {
          Two dot = 0;
          const Two r2 = two(r[n], r[n]);
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            x.get(i, n, u, a[n][u]);
            g.get(i, n, u, b[n][u]);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
              float g0, g1;                                  // rotated back
              untwo(b[n][u][k], g0, g1);
              const Two dz = two(fmaf(g1, turn.s[u][k], g0 * turn.c[u][k]), fmaf(-g0, turn.s[u][k], g1 * turn.c[u][k]));
              a[n][u][k] = mul2(a[n][u][k], r2);             // xhat
              dw[u][k] = fma2(dz, a[n][u][k], dw[u][k]);
              b[n][u][k] = mul2(dz, w[u][k]);
              dot = fma2(b[n][u][k], a[n][u][k], dot);
            }
          }
          dots[n] = both(dot);
        }
        // the step's rows are in registers: their places take the next ones
        if (i + kDepth < steps) {
          x.issue(i + kDepth);
          g.issue(i + kDepth);
        }
        copies_end();
        row_sums(dots, p.lanes);
#pragma unroll
        for (int n = 0; n < F; ++n) {
          const int h = i * F + n;
          if (h >= x.left) continue;
          const float mean = -dots[n] * p.inv_d;
          const Two m2 = two(mean, mean), r2 = two(r[n], r[n]);
#pragma unroll
          for (int u = 0; u < NU; ++u) {
#pragma unroll
            for (int k = 0; k < V / 2; ++k) a[n][u][k] = NORM ? mul2(r2, fma2(a[n][u][k], m2, b[n][u][k])) : b[n][u][k];
            if (V * p.lanes * u < x.cols) R::put(o + h * (rows * S.oh) + V * p.lanes * u, a[n][u]);
          }
        }
      }
    }
    if (p.part)
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int col = V * (sub + p.lanes * u);
        if (col < p.d)
#pragma unroll
          for (int k = 0; k < V / 2; ++k) {
            float* to = sums + (side * all + (threadIdx.x >> 5) * rows + group) * p.d + col + 2 * k;
            untwo(dw[u][k], to[0], to[1]);
          }
      }
  }
  if (!p.part) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
    const int side = i >= p.d, col = i - side * p.d;
    float v = 0.f;
    for (int n = 0; n < all; ++n) v += sums[(side * all + n) * p.d + col];
    p.part[(long long)blockIdx.x * 2 * p.d + i] = v;
  }
}

// dw[side][c] = sum over the blocks, in order: a block takes 32 columns, 32 threads
// every 32nd row of partial sums each.
__global__ void __launch_bounds__(1024) head_weight_kernel(const float* part, float* dwq, float* dwk, int blocks, int d) {
  __shared__ float s[32][33];
  await_previous();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float v = 0.f;
  if (c < 2 * d)
#pragma unroll 4
    for (int b = y; b < blocks; b += 32) v += part[(long long)b * 2 * d + c];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && c < 2 * d) {
    float t = 0.f;
#pragma unroll
    for (int n = 0; n < 32; ++n) t += s[n][x];
    float* to = c < d ? dwq : dwk;
    if (to) to[c < d ? c : c - d] = t;
  }
}

mc_status err(mc_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}
uintptr_t at(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// One operand of a call: [T, heads, d] (elements of the call's type), or `bytes` in
// one piece, aligned to `align`.
struct Operand {
  const char* name;
  const void* p;
  int64_t st, sh, heads;                          // strides in elements; 0 heads: one piece
  int64_t align, bytes;
  bool out;
  const void *in0, *in1;                          // the inputs that an output may lie on exactly
};
Operand rows_of(const char* name, const void* p, int64_t st, int64_t sh, int64_t heads, bool out = false, const void* in0 = nullptr,
                const void* in1 = nullptr) {
  return {name, heads ? p : nullptr, st, sh, heads, 0, 0, out, in0, in1};
}
Operand piece(const char* name, const void* p, int64_t align, int64_t bytes, bool out = false) {
  return {name, p, 0, 0, 0, align, bytes, out, nullptr, nullptr};
}

// Fills p with what both directions share; checks strides, alignment and overlaps
// of the operands.  `wide`: features that rows can be read and written in at a time:
// 16 bytes, a pair, or 1.
mc_status fill(const char* me, const mc_heads* h, Operand* ops, int n, Params& p, int& wide) {
  const int64_t es = h->dtype == MC_BF16 ? 2 : 4;
  wide = h->d % (16 / es) == 0 ? (int)(16 / es) : 2;
  for (int i = 0; i < n; ++i) {
    Operand& o = ops[i];
    if (!o.p) continue;
    if (at(o.p) % (o.heads ? es : o.align)) return err(MC_ERR_INVALID_ARG, "%s: %s is not aligned to its type", me, o.name);
    if (!o.heads) continue;
    if (h->T == 1) o.st = o.heads * h->d;
    if (o.heads == 1) o.sh = h->d;
    if (o.st < 0 || o.sh < 0) return err(MC_ERR_INVALID_ARG, "%s: %s has a negative stride", me, o.name);
    if (o.st >= (1ll << 40) / (h->T + 1) || o.sh >= (1ll << 40) / (o.heads + 1))
      return err(MC_ERR_UNSUPPORTED, "%s: %s has strides that are too large", me, o.name);
    for (const int w : {wide, 2, 1})
      if (at(o.p) % (w * es) == 0 && o.st % w == 0 && o.sh % w == 0) {
        wide = w < wide ? w : wide;
        break;
      }
    const int64_t st[2] = {o.st, o.sh}, ext[2] = {h->T, o.heads};
    if (o.out && !distinct_addresses(st, ext, 2, h->d))
      return err(MC_ERR_INVALID_ARG, "%s: elements of %s share addresses", me, o.name);
    o.bytes = ((h->T - 1) * o.st + (o.heads - 1) * o.sh + h->d) * es;
  }
  // an output shares memory with nothing, but for head ranges side by side in one
  // buffer (q and k of one projection: equal token strides) and the inputs of its own
  // side that it may replace
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      const Operand &a = ops[i], &b = ops[j];
      if (i == j || !a.out || !a.p || !b.p || (b.out && j < i)) continue;
      if (at(a.p) >= at(b.p) + b.bytes || at(b.p) >= at(a.p) + a.bytes) continue;
      bool fine = false;
      if (a.heads && b.heads) {
        fine = !b.out && a.p == b.p && a.st == b.st && a.sh == b.sh && a.heads == b.heads && (b.p == a.in0 || b.p == a.in1) &&
               (i ^ j) % 2 == 0;         // operands of queries and keys alternate
        if (!fine && a.st == b.st && a.st > 0) {
          const Operand &lo = at(a.p) <= at(b.p) ? a : b, &hi = at(a.p) <= at(b.p) ? b : a;
          const int64_t apart = (int64_t)((at(hi.p) - at(lo.p)) / es) % a.st;
          const int64_t wide_lo = (lo.heads - 1) * lo.sh + h->d, wide_hi = (hi.heads - 1) * hi.sh + h->d;
          fine = apart >= wide_lo && apart + wide_hi <= a.st;
        }
      }
      if (!fine) return err(MC_ERR_INVALID_ARG, "%s: %s overlaps %s", me, a.name, b.name);
    }
  p.T = (int)h->T;
  p.d = h->d;
  p.rot = h->rot;
  p.heads = h->heads_q + h->heads_k;
  p.positions = h->positions;
  p.eps = h->eps;
  p.inv_d = 1.f / (float)h->d;
  for (int k = 0; k < h->rot / 2; ++k) {
    const double turns = std::exp2(-std::log2(h->theta) * 2.0 * k / h->rot) * 0.15915494309189535;
    p.turn[k] = (unsigned long long)std::ldexp(turns - std::floor(turns), 64);
  }
  return MC_OK;
}

mc_status check_shape(const char* me, const mc_heads* h) {
  if (!h) return err(MC_ERR_INVALID_ARG, "%s: null descriptor", me);
  if (h->dtype != MC_BF16 && h->dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "%s: dtype %d", me, h->dtype);
  if (h->T < 0 || h->heads_q < 1 || h->heads_k < 0 || h->d < 2 || h->d % 2 || h->d > MC_HEAD_MAX)
    return err(MC_ERR_INVALID_ARG, "%s: T %lld, heads %d and %d, d %d (even, 2..%d)", me, (long long)h->T, h->heads_q, h->heads_k,
               h->d, MC_HEAD_MAX);
  if (h->rot < 0 || h->rot % 2 || h->rot > h->d) return err(MC_ERR_INVALID_ARG, "%s: rot %d (even, 0..d)", me, h->rot);
  if (!(h->theta > 0.0) || !std::isfinite(h->theta)) return err(MC_ERR_INVALID_ARG, "%s: theta must be finite and > 0", me);
  if (!(h->eps >= 0.f) || !std::isfinite(h->eps)) return err(MC_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", me);
  if (h->heads_q > (1 << 16) || h->heads_k > (1 << 16) || h->T > (1ll << 29) ||
      h->T * ((int64_t)h->heads_q + h->heads_k) > (1ll << 34))
    return err(MC_ERR_UNSUPPORTED, "%s: T %lld with %d and %d heads is too large", me, (long long)h->T, h->heads_q, h->heads_k);
  // theta^(-2k/rot) in turns is kept as a fraction of one: finite, and exact enough
  if (h->theta < 1e-6) return err(MC_ERR_UNSUPPORTED, "%s: theta %g below 1e-6", me, h->theta);
  return MC_OK;
}

// Lanes per row, the fewest that hold it in `parts` features each, and heads per unit of
// work: as many as leave `most` units or more, but 16 steps of the loop at most (a
// token's sines cost one or two).
void split(Params& p, int parts, int flight, long long most) {
  p.lanes = 1;
  while (p.lanes * parts < p.d) p.lanes *= 2;
  const int step = 32 / p.lanes * flight;
  int steps = 16;
  while (steps > 1 && p.T * cdiv(p.heads, steps * step) < most) steps /= 2;
  p.span = steps * step;
  for (int i = 0; i < 2; ++i) p.pieces[i] = (p.side[i].heads + p.span - 1) / p.span;
  for (int i = 0; i < 3; ++i) {
    const int n = i < 2 ? p.pieces[i] : p.pieces[0] + p.pieces[1];
    p.div_pieces[i] = make_fastdiv((uint32_t)(n > 0 ? n : 1));
  }
}

template <typename T, int V, int NU, bool WHOLE>
cudaError_t run_forward(Params& p, cudaStream_t s) {
  split(p, V * NU, kFlight, sm_count() * 32);
  const long long units = (long long)p.T * (p.pieces[0] + p.pieces[1]);
  constexpr size_t smem = WHOLE ? (size_t)kDepth * kFlight * NU * kFrontThreads * V * sizeof(T) : 0;
  const auto kernel = p.rstd ? head_norm_kernel<T, V, NU, WHOLE, true> : head_norm_kernel<T, V, NU, WHOLE, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_behind(kernel, (unsigned)cdiv(units, kFrontWarps), kFrontThreads, smem, s, p);
}
template <typename T, int V, int NU, bool WHOLE>
cudaError_t run_backward(Params& p, float* dwq, float* dwk, cudaStream_t s) {
  const int wave = sm_count() * back_blocks(NU), most = wave < kBackGrid ? wave : kBackGrid;
  split(p, V * NU, kFlight, 8ll * most * kWarps);      // some units per warp, that the last ones leave few idle
  const long long blocks = cdiv((long long)p.T * (p.pieces[0] > p.pieces[1] ? p.pieces[0] : p.pieces[1]), kWarps);
  const int grid = (int)(blocks < most ? blocks : most);
  constexpr size_t fifo = WHOLE ? (size_t)2 * kDepth * kFlight * NU * kThreads * V * sizeof(T) : 0, most_sums = 2 * kWarps * MC_HEAD_MAX * 4;
  const size_t smem = fifo + (p.part ? (size_t)2 * kWarps * (32 / p.lanes) * p.d * 4 : 0);   // a warp's rows have at most 256 features
  // the limit belongs to the kernel, not to this call: always that of the largest
  const auto kernel = p.rstd ? head_norm_back_kernel<T, V, NU, WHOLE, true> : head_norm_back_kernel<T, V, NU, WHOLE, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(fifo + most_sums));
  if (e != cudaSuccess) return e;
  e = launch_behind(kernel, (unsigned)grid, kThreads, smem, s, p);
  if (e != cudaSuccess || !p.part) return e;
  return launch_behind(head_weight_kernel, (unsigned)cdiv(2 * p.d, 32), 1024, 0, s, p.part, dwq, dwk, grid, p.d);
}

// By the features that rows can be accessed in (16 bytes, a pair, one) and the width.
template <typename F>
cudaError_t by_width(const mc_heads* h, int wide, F run) {
  using B = __nv_bfloat16;
  if (h->dtype == MC_BF16) return wide == 8 ? run.template go<B, 8, 1, true>() : wide == 2 ? run.template go<B, 2, 4, true>() : run.template go<B, 2, 4, false>();
  if (wide == 4) return h->d <= 128 ? run.template go<float, 4, 1, true>() : run.template go<float, 4, 2, true>();
  return wide == 2 ? run.template go<float, 2, 4, true>() : run.template go<float, 2, 4, false>();
}
struct Forward {
  Params& p;
  cudaStream_t s;
  template <typename T, int V, int NU, bool WHOLE>
  cudaError_t go() { return run_forward<T, V, NU, WHOLE>(p, s); }
};
struct Backward {
  Params& p;
  float *dwq, *dwk;
  cudaStream_t s;
  template <typename T, int V, int NU, bool WHOLE>
  cudaError_t go() { return run_backward<T, V, NU, WHOLE>(p, dwq, dwk, s); }
};

}  // namespace hn
}  // namespace
}  // namespace mc

using namespace mc;
using namespace mc::hn;

extern "C" {

mc_status mc_head_norm_rope(const mc_heads* h, const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                            int64_t k_head, const void* wq, const void* wk, void* yq, int64_t yq_token, int64_t yq_head,
                            void* yk, int64_t yk_token, int64_t yk_head, float* rstd, mc_stream_t stream) {
  const char* me = "mc_head_norm_rope";
  mc_status st = check_shape(me, h);
  if (st != MC_OK) return st;
  if (h->T == 0) return record_error(MC_OK, "");
  const int64_t es = h->dtype == MC_BF16 ? 2 : 4, H = h->heads_q, G = h->heads_k;
  if (h->no_norm) rstd = nullptr;
  if (!q || !yq || (!rstd && !h->no_norm) || (G && (!k || !yk))) return err(MC_ERR_INVALID_ARG, "%s: null pointer", me);
  Operand ops[] = {rows_of("q", q, q_token, q_head, H),
                   rows_of("k", k, k_token, k_head, G),
                   rows_of("yq", yq, yq_token, yq_head, H, true, q, q),
                   rows_of("yk", yk, yk_token, yk_head, G, true, k, k),
                   piece("wq", wq, es, h->d * es),
                   piece("wk", G ? wk : nullptr, es, h->d * es),
                   piece("positions", h->positions, 4, h->T * 4),
                   piece("rstd", rstd, 4, h->T * (H + G) * 4, true)};
  Params p;
  memset(&p, 0, sizeof p);
  int wide;
  if ((st = fill(me, h, ops, 8, p, wide)) != MC_OK) return st;
  if (wide > 2 && (at(wq) % 16 || (G && at(wk) % 16))) wide = 2;
  p.side[0] = {q, nullptr, yq, wq, ops[0].st, ops[0].sh, 0, 0, ops[2].st, ops[2].sh, h->heads_q};
  p.side[1] = {k, nullptr, yk, G ? wk : nullptr, ops[1].st, ops[1].sh, 0, 0, ops[3].st, ops[3].sh, h->heads_k};
  p.rstd = rstd;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = by_width(h, wide, Forward{p, s});
  if (e != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(e));
  return record_error(MC_OK, "");
}

mc_status mc_head_norm_rope_backward_workspace_size(int32_t d, size_t* bytes) {
  if (d < 2 || d % 2 || d > MC_HEAD_MAX || !bytes)
    return err(MC_ERR_INVALID_ARG, "mc_head_norm_rope_backward: d %d (even, 2..%d) or null bytes", d, MC_HEAD_MAX);
  *bytes = (size_t)kBackGrid * 2 * d * 4;
  return record_error(MC_OK, "");
}

mc_status mc_head_norm_rope_backward(const mc_heads* h, const void* dyq, int64_t dyq_token, int64_t dyq_head, const void* dyk,
                                     int64_t dyk_token, int64_t dyk_head, const void* q, int64_t q_token, int64_t q_head,
                                     const void* k, int64_t k_token, int64_t k_head, const float* rstd, const void* wq,
                                     const void* wk, void* dq, int64_t dq_token, int64_t dq_head, void* dk, int64_t dk_token,
                                     int64_t dk_head, float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
                                     mc_stream_t stream) {
  const char* me = "mc_head_norm_rope_backward";
  mc_status st = check_shape(me, h);
  if (st != MC_OK) return st;
  const cudaStream_t s = (cudaStream_t)stream;
  const int64_t es = h->dtype == MC_BF16 ? 2 : 4, H = h->heads_q, G = h->heads_k;
  if (at(dwq) % 4 || (G && at(dwk) % 4)) return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  if (h->T == 0) {                                // sums over nothing
    for (float* w : {dwq, G ? dwk : nullptr}) {
      const cudaError_t e = w ? cudaMemsetAsync(w, 0, (size_t)h->d * 4, s) : cudaSuccess;
      if (e != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(e));
    }
    return record_error(MC_OK, "");
  }
  if (h->no_norm) rstd = nullptr;
  if (!dyq || !q || (!rstd && !h->no_norm) || !dq || (G && (!dyk || !k || !dk))) return err(MC_ERR_INVALID_ARG, "%s: null pointer", me);
  const bool weights = dwq || (G && dwk);
  const size_t need = (size_t)kBackGrid * 2 * h->d * 4;
  if (weights && (!workspace || at(workspace) % 16 || workspace_bytes < need))
    return err(MC_ERR_WORKSPACE, "%s: weight gradients need a 16-byte aligned workspace of %zu bytes", me, need);
  Operand ops[] = {rows_of("dyq", dyq, dyq_token, dyq_head, H),
                   rows_of("dyk", dyk, dyk_token, dyk_head, G),
                   rows_of("q", q, q_token, q_head, H),
                   rows_of("k", k, k_token, k_head, G),
                   rows_of("dq", dq, dq_token, dq_head, H, true, dyq, q),
                   rows_of("dk", dk, dk_token, dk_head, G, true, dyk, k),
                   piece("wq", wq, es, h->d * es),
                   piece("wk", G ? wk : nullptr, es, h->d * es),
                   piece("positions", h->positions, 4, h->T * 4),
                   piece("rstd", rstd, 4, h->T * (H + G) * 4),
                   piece("dwq", dwq, 4, h->d * 4ll, true),
                   piece("dwk", G ? dwk : nullptr, 4, h->d * 4ll, true),
                   piece("workspace", weights ? workspace : nullptr, 16, (int64_t)need, true)};
  Params p;
  memset(&p, 0, sizeof p);
  int wide;
  if ((st = fill(me, h, ops, 13, p, wide)) != MC_OK) return st;
  if (wide > 2 && (at(wq) % 16 || (G && at(wk) % 16))) wide = 2;
  p.side[0] = {q, dyq, dq, wq, ops[2].st, ops[2].sh, ops[0].st, ops[0].sh, ops[4].st, ops[4].sh, h->heads_q};
  p.side[1] = {k, dyk, dk, G ? wk : nullptr, ops[3].st, ops[3].sh, ops[1].st, ops[1].sh, ops[5].st, ops[5].sh, h->heads_k};
  p.rstd = const_cast<float*>(rstd);              // read only
  p.part = weights ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e;
  float* dw = G ? dwk : nullptr;
  e = by_width(h, wide, Backward{p, dwq, dw, s});
  if (e != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(e));
  return record_error(MC_OK, "");
}

}  // extern "C"
