// RMS norm with the residual's addition, and the norm's gradient, per row of
// `cols` values (the norms between an attention block's products; the MLA
// latents' is the weightless one):
//
//   mc_add_rms_norm       h = rn(x + residual), rstd = 1 / sqrt(mean(h^2) + eps),
//                         y = h rstd w, in the inputs' type or as e4m3 with one
//                         fp32 scale per row and 128 columns:
//                         scale = max(max|y| / 448, 2^-100), q = rn(y / scale)
//   mc_rms_norm_backward  xhat = h rstd, g = w dy,
//                         dx = rstd (g - xhat mean(g xhat)) + dres,
//                         dw = sum over the rows of dy xhat
//
// Both stream each value once: a row stays in the registers of the warps that
// share it, between the sum over the row and its use.  A warp takes units of 32
// lanes x 16 bytes (or, where a pointer, pitch or width is not a multiple of 16
// bytes, of 128 single values); unit u of a row belongs to warp u mod WPR, each
// warp holds at most NU units.  Rows too wide for that (NU = 0) are read twice.
// Eight warps hold 8192 bf16 columns of the norm and 4096 of its gradient (half of
// that of fp32 or unaligned rows).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/muonclip.h"
#include "common.cuh"
#include "kernels.h"

namespace mc {
namespace {
namespace nm {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = 128;               // columns per e4m3 scale
constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 7.888609052210118e-31f;   // 2^-100: 1 / scale stays finite
constexpr int kBackGrid = 304;           // blocks of the backward (two per SM); its workspace's rows

// A lane's share of a unit: E values of the row from column col(unit, lane, 0).
template <typename T, bool VEC>
struct Unit;
template <>
struct Unit<__nv_bfloat16, true> {
  static constexpr int E = 8, kCols = 256;
  uint4 r;
  __device__ static int col(int unit, int lane, int) { return unit * kCols + lane * E; }
  __device__ void load(const __nv_bfloat16* p, int unit, int lane, int cols) {
    const int c = col(unit, lane, 0);
    r = c < cols ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0);
  }
  __device__ void get(float (&v)[E]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&v)[E]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ void store(__nv_bfloat16* p, int unit, int lane, int cols) const {
    const int c = col(unit, lane, 0);
    if (c < cols) *reinterpret_cast<uint4*>(p + c) = r;
  }
};
template <>
struct Unit<float, true> {
  static constexpr int E = 4, kCols = 128;
  float4 r;
  __device__ static int col(int unit, int lane, int) { return unit * kCols + lane * E; }
  __device__ void load(const float* p, int unit, int lane, int cols) {
    const int c = col(unit, lane, 0);
    r = c < cols ? *reinterpret_cast<const float4*>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ void get(float (&v)[E]) const { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
  __device__ void set(const float (&v)[E]) { r = make_float4(v[0], v[1], v[2], v[3]); }
  __device__ void store(float* p, int unit, int lane, int cols) const {
    const int c = col(unit, lane, 0);
    if (c < cols) *reinterpret_cast<float4*>(p + c) = r;
  }
};
template <typename T>
struct Unit<T, false> {
  static constexpr int E = 4, kCols = 128;
  T r[E];
  __device__ static int col(int unit, int lane, int e) { return unit * kCols + e * 32 + lane; }
  __device__ void load(const T* p, int unit, int lane, int cols) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = col(unit, lane, e);
      r[e] = c < cols ? p[c] : T(0.f);
    }
  }
  __device__ void get(float (&v)[E]) const {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = static_cast<float>(r[e]);
  }
  __device__ void set(const float (&v)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] = T(v[e]);
  }
  __device__ void store(T* p, int unit, int lane, int cols) const {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = col(unit, lane, e);
      if (c < cols) p[c] = r[e];
    }
  }
};

// Most units of a row per warp.
template <typename T, bool VEC>
constexpr int kAddUnits = 4;
template <typename T, bool VEC>
constexpr int kBackUnits = 2;

__device__ inline float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Packed pairs of a unit's values.
template <int E>
__device__ inline void mul_all(float (&v)[E], const float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += 2) untwo(mul2(two(v[e], v[e + 1]), two(f[e], f[e + 1])), v[e], v[e + 1]);
}
template <int E>
__device__ inline void mul_all(float (&v)[E], float f) {
  const unsigned long long f2 = two(f, f);
#pragma unroll
  for (int e = 0; e < E; e += 2) untwo(mul2(two(v[e], v[e + 1]), f2), v[e], v[e + 1]);
}

// v / f for f > 0 (or NaN): with r the rounded reciprocal, v r is at most 1.5 units
// in the last place off; adding r times the remainder v - (v r) f, which one fused
// step gives exactly, leaves the quotient's own rounding (Markstein, IBM Journal of
// Research and Development 34, 1990).  Two more packed steps per pair; the division
// operator instead takes 40.8 us for 4096 x 7168, this 34.6, the product without the
// remainder, which gives values next to a tie the neighbouring code, 33.8.
template <int E>
__device__ inline void div_all(float (&v)[E], float f) {
  const float r = __frcp_rn(f), g = -fminf(f, 3.402823466e38f);      // f = inf: v 0, not inf 0
  const unsigned long long r2 = two(r, r), g2 = two(g, g);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const unsigned long long a = two(v[e], v[e + 1]), q = mul2(a, r2);
    untwo(fma2(fma2(q, g2, a), r2, q), v[e], v[e + 1]);
  }
}

// v / f in the same way for one value and a constant; NaN and infinity stay.
__device__ inline float div_one(float v, float f) {
  const float r = 1.f / f, q = v * r;
  return v <= 3.402823466e38f ? fmaf(fmaf(q, -f, v), r, q) : v;
}

// e4m3 of a unit's values and the tiles' scales.  A 16-byte bf16 unit covers
// two tiles (a half-warp each), the others one.
template <typename T, bool VEC>
__device__ inline void store_e4m3(uint8_t* y, float* scales, int unit, int lane, int cols,
                                  float (&v)[Unit<T, VEC>::E]) {
  using U = Unit<T, VEC>;
  constexpr int lanes = 32 * kTile / U::kCols;
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < U::E; ++e) top = max_nan(top, fabsf(v[e]));
#pragma unroll
  for (int o = lanes / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float scale = max_nan(div_one(top, kE4m3Max), kScaleMin);
  const int tile0 = unit * U::kCols + (lane / lanes) * kTile;
  if (lane % lanes == 0 && tile0 < cols) scales[tile0 / kTile] = scale;
  div_all(v, scale);
  uint32_t w[(U::E + 3) / 4] = {};
#pragma unroll
  for (int e = 0; e < U::E; e += 2) {
    const uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(v[e], v[e + 1]), __NV_SATFINITE, __NV_E4M3);
    w[e / 4] = e % 4 ? __byte_perm(w[e / 4], pair, 0x5410) : pair;
  }
  if (VEC) {
    const int c = U::col(unit, lane, 0);
    if (c < cols) {
      if (U::E == 8) *reinterpret_cast<uint2*>(y + c) = make_uint2(w[0], w[(U::E + 3) / 4 - 1]);
      else *reinterpret_cast<uint32_t*>(y + c) = w[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < U::E; ++e) {
      const int c = U::col(unit, lane, e);
      if (c < cols) y[c] = (uint8_t)(w[0] >> (8 * e));
    }
  }
}

__device__ inline float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

struct AddParams {
  const void* x; const void* r; const void* w;
  void* h; void* y; float* scales; float* rstd;
  long long ldx, ldr, ldh, ldy, lds, rows;
  int cols, f8;
  float eps;
};

// The sum over the row's WPR warps of one value per lane, in a fixed order.
// red: one slot per warp; the block's threads all call it.
template <int WPR>
__device__ inline float row_sum(float s, float* red) {
  s = warp_sum(s);
  if (WPR == 1) return s;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = s;
  __syncthreads();
  const int first = warp / WPR * WPR;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) t += red[first + i];
  return t;
}

// A row per WPR warps, NU units of it per warp (0: a row of any width, read
// twice).  Widths and shares are template parameters because these kernels spend
// their time on instructions as much as on memory (a run-time WPR: 39 us for
// 4096 x 7168 with e4m3 output, 68 % of the issue slots).  Bound by memory where
// there are rows enough: that case's 206 MB in 33.8 us (6.1 TB/s); one row of it
// in 5.4 us, the latency of a load, the row's sum and two stores.
template <typename T, bool VEC, int WPR, int NU>
__global__ void __launch_bounds__(kThreads) add_norm_kernel(const __grid_constant__ AddParams p) {
  using U = Unit<T, VEC>;
  constexpr int N = NU ? NU : 1;
  __shared__ float red[kWarps];
  await_previous();
  release_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = warp % WPR;
  const long long row = (long long)blockIdx.x * (kWarps / WPR) + warp / WPR;
  const bool live = row < p.rows;
  const long long at = live ? row : 0;
  const T* x = static_cast<const T*>(p.x) + at * p.ldx;
  const T* r = p.r ? static_cast<const T*>(p.r) + at * p.ldr : nullptr;
  T* h = p.r ? static_cast<T*>(p.h) + at * p.ldh : nullptr;
  const T* w = static_cast<const T*>(p.w);
  const int cols = live ? p.cols : 0;    // rows past the end read and write nothing
  const int units = (p.cols + U::kCols - 1) / U::kCols;
  // a <- h of the unit (stored where there is a residual); its squares onto s
  unsigned long long s2 = 0;
  auto add = [&](int unit, U& a, const U& b) {
    float v[U::E];
    a.get(v);
    if (r) {
      float t[U::E];
      b.get(t);
#pragma unroll
      for (int e = 0; e < U::E; e += 2) untwo(add2(two(v[e], v[e + 1]), two(t[e], t[e + 1])), v[e], v[e + 1]);
      a.set(v);
      a.store(h, unit, lane, cols);
      a.get(v);
    }
#pragma unroll
    for (int e = 0; e < U::E; e += 2) s2 = fma2(two(v[e], v[e + 1]), two(v[e], v[e + 1]), s2);
  };
  auto finish = [&](int unit, float rs, U& a, const U& uw) {
    float v[U::E];
    a.get(v);
    mul_all(v, rs);
    if (w) {
      float f[U::E];
      uw.get(f);
      mul_all(v, f);
    }
    if (p.f8) {
      store_e4m3<T, VEC>(static_cast<uint8_t*>(p.y) + at * p.ldy, p.scales + at * p.lds, unit, lane, cols, v);
    } else {
      a.set(v);
      a.store(static_cast<T*>(p.y) + at * p.ldy, unit, lane, cols);
    }
  };
  // the row stays packed in its own type between the two uses of it
  U ux[N], ur[N];
  if (NU) {
#pragma unroll
    for (int k = 0; k < N; ++k) ux[k].load(x, k * WPR + w0, lane, cols);
    if (r) {
#pragma unroll
      for (int k = 0; k < N; ++k) ur[k].load(r, k * WPR + w0, lane, cols);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) add(k * WPR + w0, ux[k], ur[k]);
    if (w) {                             // into the residual's registers, under the sum
#pragma unroll
      for (int k = 0; k < N; ++k) ur[k].load(w, k * WPR + w0, lane, p.cols);
    }
  } else {
    for (int u = w0; u < units; u += WPR) {
      ux[0].load(x, u, lane, cols);
      if (r) ur[0].load(r, u, lane, cols);
      add(u, ux[0], ur[0]);
    }
  }
  float sa, sb;
  untwo(s2, sa, sb);
  const float s = row_sum<WPR>(sa + sb, red);
  const float rs = 1.f / sqrtf(s / (float)p.cols + p.eps);
  if (live && p.rstd && w0 == 0 && lane == 0) p.rstd[row] = rs;
  if (NU) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k * WPR + w0 < units) finish(k * WPR + w0, rs, ux[k], ur[k]);
  } else {
    const T* again = r ? h : x;          // each lane reads back its own values
    for (int u = w0; u < units; u += WPR) {
      ux[0].load(again, u, lane, cols);
      if (w) ur[0].load(w, u, lane, p.cols);
      finish(u, rs, ux[0], ur[0]);
    }
  }
}

struct BackParams {
  const void* dy; const void* h; const float* rstd; const void* w; const void* dres;
  void* dx; float* part;                 // [grid][cols] sums of dy xhat, or null
  long long lddy, ldh, ldr, ldx, rows;
  int cols;
};

// dx = rstd g - (rstd mean(g xhat)) xhat + dres and dw += dy xhat, with xhat formed
// from h both before and after the row's sum (h itself may be far from 1, so rstd
// stays with it).
// Row groups of WPR warps walk the rows in steps of grid * groups; the next row
// is loaded while the current one is worked on, both packed in their own type,
// and each lane keeps its columns' weights and sums.  The groups of a block add
// up in order through shared memory, and the block writes one row of partial
// sums.  16384 x 2048 with a weight and dres, 268 MB: 43.3 us (6.2 TB/s), plus 4.3
// for the weight's sums below.  (Loading a row at a time, with xhat and g as fp32
// arrays: 80 us.)  Rows with NU = 0 load nothing ahead, read dy and h twice and
// carry the weight's sums in global memory: 177 us for 4096 x 7168 bf16, whose 235
// MB need 35.
template <typename T, bool VEC, int WPR, int NU>
__global__ void __launch_bounds__(kThreads, 2) norm_back_kernel(const __grid_constant__ BackParams p) {
  using U = Unit<T, VEC>;
  constexpr int N = NU ? NU : 1, groups = kWarps / WPR;
  __shared__ float red[2][kWarps];
  extern __shared__ float sums[];        // [cols] when several groups share a block
  await_previous();
  release_next();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = warp % WPR, mine = warp / WPR;
  const int units = (p.cols + U::kCols - 1) / U::kCols;
  const T* w = static_cast<const T*>(p.w);
  float* part = p.part ? p.part + (long long)blockIdx.x * p.cols : nullptr;
  float acc[N][U::E] = {};
  U uw[N];
  if (NU) {
    if (w) {
#pragma unroll
      for (int k = 0; k < N; ++k) uw[k].load(w, k * WPR + w0, lane, p.cols);
    }
  } else if (part) {                     // wide rows: the block's own partial sums in global memory
    for (int c = threadIdx.x; c < p.cols; c += kThreads) part[c] = 0.f;
    __syncthreads();
  }
  // t2 += sum of w dy xhat over a unit; a += dy xhat
  auto before = [&](float rs, const U& uy, const U& uh, const U& wt, float (&a)[U::E], unsigned long long& t2) {
    float y[U::E], f[U::E];
    uh.get(y);
    mul_all(y, rs);
    uy.get(f);
    mul_all(y, f);
#pragma unroll
    for (int e = 0; e < U::E; e += 2) untwo(add2(two(y[e], y[e + 1]), two(a[e], a[e + 1])), a[e], a[e + 1]);
    if (w) {
      wt.get(f);
#pragma unroll
      for (int e = 0; e < U::E; e += 2) t2 = fma2(two(y[e], y[e + 1]), two(f[e], f[e + 1]), t2);
    } else {
#pragma unroll
      for (int e = 0; e < U::E; e += 2) t2 = add2(two(y[e], y[e + 1]), t2);
    }
  };
  // dx of a unit, given c = -rstd mean(g xhat)
  auto after = [&](T* dx, int unit, int cols, float rs, float c, const U& uy, const U& uh, const U& wt, const U& ud) {
    float v[U::E], f[U::E];
    uh.get(v);
    mul_all(v, rs);
    const unsigned long long c2 = two(c, c), r2 = two(rs, rs);
    if (p.dres) {
      ud.get(f);
#pragma unroll
      for (int e = 0; e < U::E; e += 2) untwo(fma2(two(v[e], v[e + 1]), c2, two(f[e], f[e + 1])), v[e], v[e + 1]);
    } else {
      mul_all(v, c);
    }
    float y[U::E];
    uy.get(y);
    if (w) {
      wt.get(f);
      mul_all(y, f);
    }
#pragma unroll
    for (int e = 0; e < U::E; e += 2) untwo(fma2(two(y[e], y[e + 1]), r2, two(v[e], v[e + 1])), v[e], v[e + 1]);
    U o;
    o.set(v);
    o.store(dx, unit, lane, cols);
  };
  struct Row {
    U y[N], h[N], d[N];
    float rs;
    long long at;
    int cols;
  };
  // a row past the end reads nothing and counts as zeros
  auto fetch = [&](long long row0, Row& q) {
    const long long row = row0 + mine;
    const bool live = row < p.rows;
    q.at = live ? row : 0;
    q.cols = live ? p.cols : 0;
    q.rs = live ? p.rstd[row] : 0.f;
    if (!NU) return;
    const T* dy = static_cast<const T*>(p.dy) + q.at * p.lddy;
    const T* h = static_cast<const T*>(p.h) + q.at * p.ldh;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      q.y[k].load(dy, k * WPR + w0, lane, q.cols);
      q.h[k].load(h, k * WPR + w0, lane, q.cols);
    }
    if (p.dres) {
      const T* dres = static_cast<const T*>(p.dres) + q.at * p.ldr;
#pragma unroll
      for (int k = 0; k < N; ++k) q.d[k].load(dres, k * WPR + w0, lane, q.cols);
    }
  };
  const long long step = (long long)gridDim.x * groups;
  const float inv_n = 1.f / (float)p.cols;
  int turn = 0;
  Row now, next;
  fetch((long long)blockIdx.x * groups, now);
  for (long long row0 = (long long)blockIdx.x * groups; row0 < p.rows; row0 += step, turn ^= 1) {
    fetch(row0 + step, next);
    T* dx = static_cast<T*>(p.dx) + now.at * p.ldx;
    const float rs = now.rs;
    unsigned long long t2 = 0;
    float ta, tb;
    if (NU) {
#pragma unroll
      for (int k = 0; k < N; ++k) before(rs, now.y[k], now.h[k], uw[k], acc[k], t2);
      untwo(t2, ta, tb);
      const float c = -rs * (row_sum<WPR>(ta + tb, red[turn]) * inv_n);
#pragma unroll
      for (int k = 0; k < N; ++k) after(dx, k * WPR + w0, now.cols, rs, c, now.y[k], now.h[k], uw[k], now.d[k]);
    } else {
      const T* dy = static_cast<const T*>(p.dy) + now.at * p.lddy;
      const T* h = static_cast<const T*>(p.h) + now.at * p.ldh;
      for (int u = w0; u < units; u += WPR) {
        now.y[0].load(dy, u, lane, now.cols);
        now.h[0].load(h, u, lane, now.cols);
        if (w) uw[0].load(w, u, lane, p.cols);
        float a[U::E] = {};
        before(rs, now.y[0], now.h[0], uw[0], a, t2);
#pragma unroll
        for (int e = 0; e < U::E; ++e) {
          const int c = U::col(u, lane, e) + (VEC ? e : 0);
          if (part && c < now.cols) part[c] += a[e];
        }
      }
      untwo(t2, ta, tb);
      const float c = -rs * (row_sum<WPR>(ta + tb, red[turn]) * inv_n);
      for (int u = w0; u < units; u += WPR) {
        now.y[0].load(dy, u, lane, now.cols);
        now.h[0].load(h, u, lane, now.cols);
        if (w) uw[0].load(w, u, lane, p.cols);
        if (p.dres) now.d[0].load(static_cast<const T*>(p.dres) + now.at * p.ldr, u, lane, now.cols);
        after(dx, u, now.cols, rs, c, now.y[0], now.h[0], uw[0], now.d[0]);
      }
    }
    now = next;
  }
  if (!NU || !part) return;
  for (int gr = groups - 1; gr >= 0; --gr) {
    if (gr == mine) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int e = 0; e < U::E; ++e) {
          const int c = U::col(k * WPR + w0, lane, e) + (VEC ? e : 0);
          if (c >= p.cols) continue;
          const float t = (gr == groups - 1 ? 0.f : sums[c]) + acc[k][e];
          if (gr) sums[c] = t;
          else part[c] = t;
        }
    }
    if (groups > 1) __syncthreads();
  }
}

// dw[c] = sum over the partial rows: 32 columns per block, a warp per 32nd row,
// the 32 sums added in a fixed tree.  Latency: 4.3 us for 2.5 MB (2048 columns).
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* part, float* dw, int n, int cols) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  await_previous();
  constexpr int flight = (kBackGrid + 31) / 32;        // every load at once
  float v[flight];
#pragma unroll
  for (int k = 0; k < flight; ++k) {
    const int i = warp + 32 * k;
    v[k] = c < cols && i < n ? part[(long long)i * cols + c] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < flight; ++k) s += v[k];
  red[warp][lane] = s;
  __syncthreads();
  s = red[lane][warp];                   // a warp per column now
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int d = blockIdx.x * 32 + warp;
  if (lane == 0 && d < cols) dw[d] = s;
}

// The fewest warps that hold a row of `cols` in at most MOST units each, as
// f(WPR, NU); NU = 0 when eight cannot.
template <int W, int N>
struct Share {};
template <int MOST, typename F>
cudaError_t by_share(int cols, int unit_cols, F f) {
  const int units = (cols + unit_cols - 1) / unit_cols;
  if (units <= 1) return f(Share<1, 1>());
  if (units <= MOST) return f(Share<1, MOST>());
  if (units <= 2 * MOST) return f(Share<2, MOST>());
  if (units <= 4 * MOST) return f(Share<4, MOST>());
  if (units <= 8 * MOST) return f(Share<8, MOST>());
  return f(Share<8, 0>());
}

template <typename T, bool VEC>
struct AddLaunch {
  const AddParams& p;
  cudaStream_t s;
  template <int WPR, int NU>
  cudaError_t operator()(Share<WPR, NU>) const {
    return launch_behind(add_norm_kernel<T, VEC, WPR, NU>, (unsigned)cdiv(p.rows, kWarps / WPR), kThreads, 0, s, p);
  }
};
template <typename T, bool VEC>
cudaError_t launch_add(const AddParams& p, cudaStream_t s) {
  return by_share<kAddUnits<T, VEC>>(p.cols, Unit<T, VEC>::kCols, AddLaunch<T, VEC>{p, s});
}

template <typename T, bool VEC>
struct BackLaunch {
  const BackParams& p;
  int& grid;
  cudaStream_t s;
  template <int WPR, int NU>
  cudaError_t operator()(Share<WPR, NU>) const {
    constexpr int groups = kWarps / WPR;
    const long long want = cdiv(p.rows, groups);
    grid = (int)(want < kBackGrid ? want : kBackGrid);
    const size_t smem = p.part && groups > 1 && NU ? (size_t)p.cols * 4 : 0;   // at most 2048 columns: 8 KB
    return launch_behind(norm_back_kernel<T, VEC, WPR, NU>, (unsigned)grid, kThreads, smem, s, p);
  }
};
template <typename T, bool VEC>
cudaError_t launch_back(const BackParams& p, float* dw, cudaStream_t s) {
  int grid = 0;
  const cudaError_t e = by_share<kBackUnits<T, VEC>>(p.cols, Unit<T, VEC>::kCols, BackLaunch<T, VEC>{p, grid, s});
  if (e != cudaSuccess || !p.part) return e;
  return launch_behind(norm_weight_kernel, (unsigned)cdiv(p.cols, 32), 1024, 0, s, p.part, dw, grid, p.cols);
}

mc_status err(mc_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}

// One 2-D operand of a call: rows of `bytes` bytes each `pitch` bytes apart.
struct Rows {
  const char* name;
  const void* p;
  long long pitch, bytes;
  bool out;
};
uintptr_t at(const Rows& a) { return reinterpret_cast<uintptr_t>(a.p); }
// Whether two operands of `n` rows share an address.  Equal pitches allow two
// column ranges of one buffer.
bool overlap(const Rows& a, const Rows& b, long long n) {
  const uintptr_t ea = at(a) + (n - 1) * a.pitch + a.bytes, eb = at(b) + (n - 1) * b.pitch + b.bytes;
  if (at(a) >= eb || at(b) >= ea) return false;
  if (a.pitch != b.pitch || a.pitch == 0 || n == 1) return true;
  const Rows &lo = at(a) <= at(b) ? a : b, &hi = at(a) <= at(b) ? b : a;
  const long long d = (long long)((at(hi) - at(lo)) % (uintptr_t)a.pitch);
  return d < lo.bytes || d + hi.bytes > a.pitch;
}
// Outputs may lie exactly on an operand that `same` allows, and share no
// address with any other.
template <typename Same>
mc_status check_overlaps(const char* call, const Rows* t, int n, long long rows, Same same) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (i == j || !t[i].out || !t[i].p || !t[j].p || (t[j].out && j < i)) continue;
      if (same(i, j) && t[i].p == t[j].p && t[i].pitch == t[j].pitch) continue;
      if (overlap(t[i], t[j], rows)) return err(MC_ERR_INVALID_ARG, "%s: %s overlaps %s", call, t[i].name, t[j].name);
    }
  return MC_OK;
}
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace nm
}  // namespace
}  // namespace mc

using namespace mc;
using namespace mc::nm;

extern "C" {

mc_status mc_add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                          void* h, int64_t ldh, void* y, int64_t ldy, float* scales, int64_t lds, float* rstd,
                          int64_t rows, int32_t cols, int32_t dtype, int32_t y_dtype, float eps,
                          mc_stream_t stream) {
  const char* me = "mc_add_rms_norm";
  if (dtype != MC_BF16 && dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "%s: dtype %d", me, dtype);
  if (y_dtype != dtype && y_dtype != MC_F8E4M3) return err(MC_ERR_INVALID_ARG, "%s: y_dtype %d", me, y_dtype);
  const bool f8 = y_dtype == MC_F8E4M3;
  if (rows < 0 || rows > 0x7fffffff || cols < 1 || cols > (1 << 30))
    return err(MC_ERR_INVALID_ARG, "%s: rows %lld, cols %d", me, (long long)rows, cols);
  const int tiles = (cols + kTile - 1) / kTile;
  if (ldx < cols || ldy < cols || (residual && (ldr < cols || ldh < cols)) || (f8 && scales && lds < tiles))
    return err(MC_ERR_INVALID_ARG, "%s: a pitch is below its row's length", me);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return err(MC_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", me);
  if (rows == 0) return record_error(MC_OK, "");
  if ((residual == nullptr) != (h == nullptr)) return err(MC_ERR_INVALID_ARG, "%s: residual and h go together", me);
  if (f8 != (scales != nullptr)) return err(MC_ERR_INVALID_ARG, "%s: scales go with an e4m3 y", me);
  if (!x || !y) return err(MC_ERR_INVALID_ARG, "%s: null pointer", me);
  const size_t es = dtype == MC_BF16 ? 2 : 4;
  for (const void* p : {x, residual, weight, static_cast<const void*>(h), static_cast<const void*>(f8 ? nullptr : y)})
    if (!aligned(p, es)) return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  if (!aligned(scales, 4) || !aligned(rstd, 4)) return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  const long long e = (long long)es;
  const Rows t[] = {{"x", x, ldx * e, cols * e, false},
                    {"residual", residual, ldr * e, cols * e, false},
                    {"weight", weight, 0, cols * e, false},
                    {"h", h, ldh * e, cols * e, true},
                    {"y", y, ldy * (f8 ? 1 : e), cols * (f8 ? 1 : e), true},
                    {"scales", scales, lds * 4, tiles * 4ll, true},
                    {"rstd", rstd, 4, 4, true}};
  // a lane writes h and y over values of x and residual that it has read
  const mc_status st = check_overlaps(me, t, 7, rows, [&](int i, int j) {
    return (i == 3 && j <= 1) || (i == 4 && j <= 1 && !f8);
  });
  if (st != MC_OK) return st;
  AddParams p{x, residual, weight, h, y, f8 ? scales : nullptr, rstd, ldx, ldr, ldh, ldy, lds, rows, cols, f8, eps};
  const int per = 16 / (int)es;          // values per 16 bytes
  const bool vec = cols % per == 0 && ldx % per == 0 && aligned(x, 16) && aligned(weight, 16) &&
                   (!residual || (ldr % per == 0 && ldh % per == 0 && aligned(residual, 16) && aligned(h, 16))) &&
                   ldy % per == 0 && aligned(y, f8 ? per : 16);
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t c;
  if (dtype == MC_BF16) c = vec ? launch_add<__nv_bfloat16, true>(p, s) : launch_add<__nv_bfloat16, false>(p, s);
  else c = vec ? launch_add<float, true>(p, s) : launch_add<float, false>(p, s);
  if (c != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(c));
  return record_error(MC_OK, "");
}

mc_status mc_rms_norm_backward_workspace_size(int32_t cols, size_t* bytes) {
  if (cols < 1 || cols > (1 << 30) || !bytes) return err(MC_ERR_INVALID_ARG, "mc_rms_norm_backward: cols %d or null bytes", cols);
  *bytes = (size_t)kBackGrid * (size_t)cols * 4;
  return record_error(MC_OK, "");
}

mc_status mc_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const float* rstd,
                               const void* weight, const void* dres, int64_t ldr, void* dx, int64_t lddx,
                               float* dweight, int64_t rows, int32_t cols, int32_t dtype, void* workspace,
                               size_t workspace_bytes, mc_stream_t stream) {
  const char* me = "mc_rms_norm_backward";
  if (dtype != MC_BF16 && dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "%s: dtype %d", me, dtype);
  if (rows < 0 || rows > 0x7fffffff || cols < 1 || cols > (1 << 30))
    return err(MC_ERR_INVALID_ARG, "%s: rows %lld, cols %d", me, (long long)rows, cols);
  if (lddy < cols || ldh < cols || lddx < cols || (dres && ldr < cols))
    return err(MC_ERR_INVALID_ARG, "%s: a pitch is below its row's length", me);
  if (!aligned(dweight, 4)) return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  const cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {                       // a sum over no rows
    const cudaError_t c = dweight ? cudaMemsetAsync(dweight, 0, (size_t)cols * 4, s) : cudaSuccess;
    if (c != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(c));
    return record_error(MC_OK, "");
  }
  if (!dy || !h || !rstd || !dx) return err(MC_ERR_INVALID_ARG, "%s: null pointer", me);
  const size_t es = dtype == MC_BF16 ? 2 : 4;
  for (const void* p : {dy, h, weight, dres, static_cast<const void*>(dx)})
    if (!aligned(p, es)) return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  if (!aligned(rstd, 4)) return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  const size_t need = (size_t)kBackGrid * (size_t)cols * 4;
  if (dweight && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return err(MC_ERR_WORKSPACE, "%s: dweight needs a 16-byte aligned workspace of %zu bytes", me, need);
  const long long e = (long long)es;
  const Rows t[] = {{"dy", dy, lddy * e, cols * e, false}, {"h", h, ldh * e, cols * e, false},
                    {"dres", dres, ldr * e, cols * e, false}, {"rstd", rstd, 4, 4, false},
                    {"weight", weight, 0, cols * e, false}, {"dx", dx, lddx * e, cols * e, true},
                    {"dweight", dweight, 0, cols * 4ll, true},
                    {"workspace", dweight ? workspace : nullptr, 0, (long long)need, true}};
  // a lane writes dx over values of dy, h and dres that it has read
  const mc_status st = check_overlaps(me, t, 8, rows, [](int i, int j) { return i == 5 && j <= 2; });
  if (st != MC_OK) return st;
  BackParams p{dy, h, rstd, weight, dres, dx, dweight ? static_cast<float*>(workspace) : nullptr,
               lddy, ldh, ldr, lddx, rows, cols};
  const int per = 16 / (int)es;
  const bool vec = cols % per == 0 && lddy % per == 0 && ldh % per == 0 && lddx % per == 0 && aligned(dy, 16) &&
                   aligned(h, 16) && aligned(dx, 16) && aligned(weight, 16) &&
                   (!dres || (ldr % per == 0 && aligned(dres, 16)));
  cudaError_t c;
  if (dtype == MC_BF16) c = vec ? launch_back<__nv_bfloat16, true>(p, dweight, s) : launch_back<__nv_bfloat16, false>(p, dweight, s);
  else c = vec ? launch_back<float, true>(p, dweight, s) : launch_back<float, false>(p, dweight, s);
  if (c != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(c));
  return record_error(MC_OK, "");
}

}  // extern "C"
