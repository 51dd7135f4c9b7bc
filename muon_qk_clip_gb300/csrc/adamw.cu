// AdamW over many tensors in one launch: the step of the parameters that Muon
// leaves out (embeddings, output tables, norm weights; [K2-notes] 3.2 applies
// Muon to the matrices of the layers).  Per value, in fp32:
//
//   m <- beta1 m + (1 - beta1) g          v <- beta2 v + (1 - beta2) g^2
//   p <- p - lr (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay p)
//
// 8-bit states hold m and r = sqrt(v) as e4m3 with one fp32 scale per 128 values
// of a tensor: scale = max(max|x| * (1 / 448), 2^-100), code = e4m3(x * (1 / scale)).
// The root is stored, not v: it is what divides, and e4m3's 2^-9 .. 448 then
// spans 2^35 of v within a block, at 2^-4 of the root.  A root above zero never
// becomes zero (the least code is 2^-9) while its square is in fp32's range, from 2^-74 up:
// a forgotten v would divide its next gradient by eps alone.  The parameter's step takes
// m and v before their rounding.  A code moves only when a step changes its value by half the way to the
// next one, 3.1 to 5.6 %: beta2 = 0.95 lowers a root by 2.5 % at most, and v follows its
// gradients because the blocks' scales, and with them the codes' places, vary from step
// to step; larger betas are refused.
//
// One pass over memory, 22 bytes a value with bf16 p and g and fp32 states, 10.1
// with 8-bit ones: 2 x 65536 x 2048 values 833 us, 7.1 TB/s (a copy reaches 6.8;
// 55 % are reads), 2 x 65521 x 2048 with 8-bit states 411 us, 6.6 TB/s (of four
// values a thread twice that).  A block takes a chunk of one tensor and finds which by a
// search over the chunks' prefix sums among the launch's parameters.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <vector>

#include "../../include/muonclip.h"
#include "common.cuh"
#include "kernels.h"

namespace mc {
namespace {
namespace aw {

// Small blocks leave their places to the next as their warps end.  (2^27 values, bf16, 8-bit
// states: five blocks of 128 threads per SM 211 us, four 228, six, with spills, 245, two
// of 256 230; fp32 states 419 and, with 256 threads, 423.)
constexpr int kThreads = 128;
// Blocks per SM with 8-bit states, by the operands' size: five leave 96 registers a thread, of which
// 16 fp32 values in flight spill.  (2^27 values, five and four blocks: bf16 parameters and gradients
// 211 and 228 us; bf16 parameters with fp32 gradients 235 to 267, as the spills fall, and 239; fp32
// parameters 303 and 281, 341 and 311.)
__host__ __device__ constexpr int blocks8(int bytes) { return bytes == 4 ? 5 : 4; }
constexpr int kBlock = MC_ADAMW_BLOCK;            // values per scale of an 8-bit state
// Values of a thread's step: four with fp32 states; 16 with 8-bit ones, so that a
// thread's codes are 16 bytes, and eight threads hold a block.
constexpr int kWide = 4, kWide8 = 16;
static_assert(kBlock == 8 * kWide8, "eight threads hold a block");
// Steps per thread block (together a chunk of a tensor) at most, so that few loads stand
// at a block's start with nothing before them, and the thread blocks that every SM has
// left with them: else fewer steps.  (Blocks of 256 threads, 2^24 and 2^25 values with 8-bit
// states: 34 and 64 us with four blocks left, 35 and 64 with two, 42 and 70 with 16; one step
// for all of 2^26 took 165.  More than 8 steps, or 4, gain nothing.)
constexpr int kSteps = 4, kSteps8 = 8, kPerSm = 8;
constexpr int kAhead = 2;                         // steps in flight with fp32 states
constexpr float kLeast = 0x1p-9f;                 // least positive e4m3
constexpr float kScaleMin = 0x1p-100f;

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  long long n;
  uint32_t begin;                                 // its first chunk
  uint32_t vec;                                   // every operand aligned to its accesses
};
struct Coef {
  float b1, c1, b2, c2;                           // beta1, 1 - beta1, beta2, 1 - beta2
  float one;                                      // 1
  float lr, wd, eps;
  float i1, i2;                                   // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float l1[2], l2[2];                             // log beta1, log beta2 in two parts (for a step on the device)
  const long long* step;                          // or null
  const float* grad_scale;                        // or null
  int32_t* status;
};
template <int N>
struct Launch {
  Tensor t[N];
  Coef c;
  int count;
  int steps;                                      // per chunk
};

using Two = unsigned long long;                   // two fp32, for one instruction on both
// Four neighbouring values.
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 w;
  __device__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ void part(const float* p, int n) {
    w = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
  }
  __device__ void get(Two (&x)[2]) const { x[0] = two(w.x, w.y); x[1] = two(w.z, w.w); }
  __device__ void set(const Two (&x)[2]) {
    untwo(x[0], w.x, w.y);
    untwo(x[1], w.z, w.w);
  }
  __device__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ void put(float* p, int n) const {
    if (n > 0) p[0] = w.x;
    if (n > 1) p[1] = w.y;
    if (n > 2) p[2] = w.z;
    if (n > 3) p[3] = w.w;
  }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 w;
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ void part(const __nv_bfloat16* p, int n) {
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = i < n ? __bfloat16_as_ushort(p[i]) : 0u;
    w = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
  }
  __device__ void get(Two (&x)[2]) const {
    x[0] = two(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
    x[1] = two(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  __device__ void set(const Two (&x)[2]) {
    float e[4];
    untwo(x[0], e[0], e[1]);
    untwo(x[1], e[2], e[3]);
    const __nv_bfloat162 a = __floats2bfloat162_rn(e[0], e[1]), b = __floats2bfloat162_rn(e[2], e[3]);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ void put(__nv_bfloat16* p, int n) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = __ushort_as_bfloat16((unsigned short)((i < 2 ? w.x : w.y) >> (16 * (i & 1))));
  }
};
// Four e4m3 codes to and from fp32.
__device__ inline void decode(uint32_t w, Two (&x)[2]) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 u = __half22float2(__half2(a)), v = __half22float2(__half2(b));
  x[0] = two(u.x, u.y);
  x[1] = two(v.x, v.y);
}
__device__ inline uint32_t encode(const float (&x)[4]) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3) << 16;
}
// 32 bytes at a time (aligned so).
__device__ inline void load_32b(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ inline void store_32b(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 16 neighbouring values, as they lie in memory.
template <typename T>
struct Row;
template <>
struct Row<float> {
  uint32_t w[16];
  __device__ void load(const float* p) { load_32b(p, w); load_32b(p + 8, w + 8); }
  __device__ void part(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
  }
  __device__ void get(int u, Two (&x)[2]) const {        // values 4 u .. 4 u + 3
    x[0] = two(__uint_as_float(w[4 * u]), __uint_as_float(w[4 * u + 1]));
    x[1] = two(__uint_as_float(w[4 * u + 2]), __uint_as_float(w[4 * u + 3]));
  }
  __device__ Four<float> four(int u) const {
    return {make_float4(__uint_as_float(w[4 * u]), __uint_as_float(w[4 * u + 1]), __uint_as_float(w[4 * u + 2]), __uint_as_float(w[4 * u + 3]))};
  }
  __device__ void set(int u, const Two (&x)[2]) {
    float e[4];
    untwo(x[0], e[0], e[1]);
    untwo(x[1], e[2], e[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * u + i] = __float_as_uint(e[i]);
  }
  __device__ void store(float* p) const { store_32b(p, w); store_32b(p + 8, w + 8); }
  __device__ void put(float* p, int n) const {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = __uint_as_float(w[i]);
  }
};
template <>
struct Row<__nv_bfloat16> {
  uint32_t w[8];
  __device__ void load(const __nv_bfloat16* p) { load_32b(p, w); }
  __device__ void part(const __nv_bfloat16* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = (2 * i < n ? (uint32_t)__bfloat16_as_ushort(p[2 * i]) : 0u) |
             (2 * i + 1 < n ? (uint32_t)__bfloat16_as_ushort(p[2 * i + 1]) << 16 : 0u);
  }
  __device__ void get(int u, Two (&x)[2]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = two(__uint_as_float(w[2 * u + i] << 16), __uint_as_float(w[2 * u + i] & 0xffff0000u));
  }
  __device__ Four<__nv_bfloat16> four(int u) const { return {make_uint2(w[2 * u], w[2 * u + 1])}; }
  __device__ void set(int u, const Two (&x)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b;
      untwo(x[i], a, b);
      const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
      w[2 * u + i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  __device__ void store(__nv_bfloat16* p) const { store_32b(p, w); }
  __device__ void put(__nv_bfloat16* p, int n) const {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = __ushort_as_bfloat16((unsigned short)(w[i / 2] >> (16 * (i & 1))));
  }
};
struct CodeRow {
  uint32_t w[4];
  __device__ void load(const uint8_t* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
  __device__ void part(const uint8_t* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
  }
  __device__ void store(uint8_t* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ void put(uint8_t* p, int n) const {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
  }
};
// Codes of the 128 values that eight neighbouring threads hold, and their scale.
// Every operation is one rounding of its operands' (no contraction), so equal states
// give equal codes wherever they are computed so.
template <bool ROOT>
__device__ inline void encode(const Two (&v)[8], CodeRow& code, float& scale) {
  auto max_nan = [](float a, float b) {            // NaN if one is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  };
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    untwo(v[i], a, b);
    top = max_nan(top, max_nan(fabsf(a), fabsf(b)));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float q = __fmul_rn(top, 1.f / 448.f);
  scale = q < kScaleMin ? kScaleMin : q;           // NaN stays NaN, as fmaxf would not let it
  const float inv = __frcp_rn(scale);
  const Two i2 = two(inv, inv);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float x[4];
    untwo(mul2(v[2 * u], i2), x[0], x[1]);
    untwo(mul2(v[2 * u + 1], i2), x[2], x[3]);
    if (ROOT) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = x[i] > 0.f ? fmaxf(x[i], kLeast) : x[i];
    }
    code.w[u] = encode(x);
  }
}

// What a thread block does: its chunk of one tensor, and the step's factors.
struct Chunk {
  long long first;                                 // the chunk's first value
  int n;                                           // its values
  float i1, i2, gs;
};
template <int N>
__device__ inline const Tensor& chunk_of(const Launch<N>& a, int step_values, Chunk& c) {
  // the last tensor whose first chunk is at or before this block
  int lo = 0;
#pragma unroll
  for (int step = N > 256 ? 256 : N / 2; step > 0; step >>= 1)      // N is 504 or a power of two
    if (lo + step < a.count && a.t[lo + step].begin <= blockIdx.x) lo += step;
  const Tensor& t = a.t[lo];
  const int chunk = a.steps * step_values;
  c.first = (long long)(blockIdx.x - t.begin) * chunk;
  c.n = (int)min(t.n - c.first, (long long)chunk);
  return t;
}
// 1 - beta^t = -expm1(t log beta), the exponent in two fp32 parts: its rest of 2^-24 and less moves
// the result by (1 + expm1) times that.  Within 2 ulp of the exact value.
__device__ inline float one_minus_power(long long t, const float (&l)[2]) {
  const float th = (float)t, tl = (float)(t - (long long)th);
  const float y = th * l[0], r = fmaf(th, l[0], -y) + fmaf(th, l[1], tl * l[0]), e = expm1f(y);
  return -fmaf(r, 1.f + e, e);
}
// The step's factors.  With a step on the device one thread of the block works its two out, in fp32.
// (2^27 values in bf16: 418 us with 32-bit states and 212 with 8-bit ones, as with a step from the
// host; every thread for itself in fp64 702 and 234.)  With 8-bit states they stand behind the block's first
// loads (in front of them 216), with 32-bit ones in front (behind them 122 vectors of 7168, with a step
// from the host, took 4.0 us of a graph instead of 3.6).
__device__ inline void factors(const Coef& a, Chunk& c) {
  c.gs = a.grad_scale ? *a.grad_scale : 1.f;
  c.i1 = a.i1;
  c.i2 = a.i2;
  if (a.step) {
    __shared__ float both[2];
    if (threadIdx.x == 0) {
      const long long t = min(max(*a.step, 1ll), 1ll << 61);      // by then a power of a beta below 1 - 2^-53 is 0
      both[0] = __frcp_rn(one_minus_power(t, a.l1));
      both[1] = __frcp_rn(__fsqrt_rn(one_minus_power(t, a.l2)));
    }
    __syncthreads();
    c.i1 = both[0];
    c.i2 = both[1];
  }
}
__device__ inline Two dup(float x) { return two(x, x); }
// Two values' step: p, m and v become the new ones, r the root of v.  m and v by
// operations of one rounding each, as encode.  (The sum of two packed products, written
// as one, is contracted to an fma, which turned a code in 10^6 against operations of
// one rounding each; a factor of 1 that the compiler does not know keeps it apart.
// Scalar sums took 3 us of 453 more, 2 x 65521 x 2048 values.)
__device__ inline void update(const Coef& c, const Chunk& k, Two g, Two& p, Two& m, Two& v, Two& r) {
  g = mul2(g, dup(k.gs));
  m = fma2(mul2(m, dup(c.b1)), dup(c.one), mul2(g, dup(c.c1)));
  v = fma2(mul2(v, dup(c.b2)), dup(c.one), mul2(mul2(g, g), dup(c.c2)));
  float v0, v1, d0, d1, m0, m1;
  untwo(v, v0, v1);
  r = two(__fsqrt_rn(v0), __fsqrt_rn(v1));
  // the quotient is of the order of 1 and moves p by lr of itself: an ulp or two of it
  // are nothing beside p's own rounding
  untwo(fma2(r, dup(k.i2), dup(c.eps)), d0, d1);
  untwo(mul2(m, dup(k.i1)), m0, m1);
  const Two u = two(__fdividef(m0, d0), __fdividef(m1, d1));
  p = fma2(dup(-c.lr), fma2(dup(c.wd), p, u), p);
}
// Zeros, or NaN once one of the values added is not finite: of four stored values, so after their
// rounding (to bf16 it may take the largest to infinity), the first n.
template <typename P>
struct Finite;
template <>
struct Finite<float> {
  Two z = 0;
  __device__ void add(const Four<float>& x, int n) {
    if (n >= 4) z = fma2(two(x.w.x, x.w.y), 0, fma2(two(x.w.z, x.w.w), 0, z));
    else z = fma2(two(n > 0 ? x.w.x : 0.f, n > 1 ? x.w.y : 0.f), 0, fma2(two(n > 2 ? x.w.z : 0.f, 0.f), 0, z));
  }
  __device__ bool all() const {
    float a, b;
    untwo(z, a, b);
    return a == 0.f && b == 0.f;
  }
};
template <>
struct Finite<__nv_bfloat16> {
  __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
  __device__ void add(const Four<__nv_bfloat16>& x, int n) {
    uint2 w = x.w;
    if (n < 4) w = make_uint2(n >= 2 ? w.x : n == 1 ? w.x & 0xffffu : 0u, n == 3 ? w.y & 0xffffu : 0u);
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.x), zero, __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.y), zero, z));
  }
  __device__ bool all() const { return __low2float(z) == 0.f && __high2float(z) == 0.f; }
};

template <typename P, typename G, int N>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Launch<N> a) {
  await_previous();
  release_next();
  Chunk k;
  constexpr int kSet = kThreads * kWide;
  const Tensor& t = chunk_of(a, kSet, k);
  factors(a.c, k);
  P* p = static_cast<P*>(t.p) + k.first;
  const G* g = static_cast<const G*>(t.g) + k.first;
  float *m = static_cast<float*>(t.m) + k.first, *v = static_cast<float*>(t.v) + k.first;
  const int n = k.n;
  const bool vec = t.vec;
  Finite<P> z;
  struct Raw {
    Four<P> p;
    Four<G> g;
    Four<float> m, v;
  } raw[kAhead];
  auto load = [&](int i, Raw& r) {
    if (vec && i + 4 <= n) {
      r.p.load(p + i);
      r.g.load(g + i);
      r.m.load(m + i);
      r.v.load(v + i);
    } else {
      r.p.part(p + i, n - i);
      r.g.part(g + i, n - i);
      r.m.part(m + i, n - i);
      r.v.part(v + i, n - i);
    }
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) load((s * kThreads + threadIdx.x) * kWide, raw[s]);
  for (int s0 = 0; s0 < a.steps; s0 += kAhead) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int i = ((s0 + s) * kThreads + threadIdx.x) * kWide;
      if (i >= n) break;
      const Raw now = raw[s];
      if (s0 + s + kAhead < a.steps) load(i + kAhead * kSet, raw[s]);
      Two pv[2], gv[2], mv[2], vv[2], rv;
      now.p.get(pv);
      now.g.get(gv);
      now.m.get(mv);
      now.v.get(vv);
#pragma unroll
      for (int x = 0; x < 2; ++x) update(a.c, k, gv[x], pv[x], mv[x], vv[x], rv);
      Four<P> np;
      Four<float> nm, nv;
      np.set(pv);
      z.add(np, n - i);
      nm.set(mv);
      nv.set(vv);
      if (vec && i + 4 <= n) {
        np.store(p + i);
        nm.store(m + i);
        nv.store(v + i);
      } else {
        np.put(p + i, n - i);
        nm.put(m + i, n - i);
        nv.put(v + i, n - i);
      }
    }
  }
  if (!z.all()) set_status(a.c.status, MC_STATUS_NONFINITE_UPDATE);
}

// The same with 8-bit states.
template <typename P, typename G, int N>
__global__ void __launch_bounds__(kThreads, blocks8(sizeof(P) + sizeof(G))) adamw8_kernel(const __grid_constant__ Launch<N> a) {
  await_previous();
  release_next();
  Chunk k;
  constexpr int kSet = kThreads * kWide8;
  const Tensor& t = chunk_of(a, kSet, k);
  P* p = static_cast<P*>(t.p) + k.first;
  const G* g = static_cast<const G*>(t.g) + k.first;
  uint8_t *m = static_cast<uint8_t*>(t.m) + k.first, *v = static_cast<uint8_t*>(t.v) + k.first;
  float *ms = t.ms + k.first / kBlock, *vs = t.vs + k.first / kBlock;
  const int n = k.n;
  const bool vec = t.vec;
  Finite<P> z;
  struct Raw {
    Row<P> p;
    Row<G> g;
    CodeRow m, v;
    float ms, vs;
  } raw;
  auto load = [&](int i) {
    if (vec && i + kWide8 <= n) {
      raw.p.load(p + i);
      raw.g.load(g + i);
      raw.m.load(m + i);
      raw.v.load(v + i);
    } else {
      raw.p.part(p + i, n - i);
      raw.g.part(g + i, n - i);
      raw.m.part(m + i, n - i);
      raw.v.part(v + i, n - i);
    }
    raw.ms = raw.vs = 0.f;
    if ((i & ~(kBlock - 1)) < n) {
      raw.ms = ms[i / kBlock];
      raw.vs = vs[i / kBlock];
    }
  };
  load(threadIdx.x * kWide8);
  factors(a.c, k);
  for (int s = 0; s < a.steps; ++s) {
    const int i = (s * kThreads + threadIdx.x) * kWide8;
    if ((s * kThreads + (threadIdx.x & ~31)) * kWide8 >= n) break;    // the whole warp is behind the end
    Raw now = raw;
    if (s + 1 < a.steps) load(i + kSet);
    Two mv[8], rv[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      Two pv[2], gv[2], m2[2], r2[2];
      now.p.get(u, pv);
      now.g.get(u, gv);
      decode(now.m.w[u], m2);
      decode(now.v.w[u], r2);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mv[2 * u + x] = mul2(m2[x], dup(now.ms));
        Two r = mul2(r2[x], dup(now.vs)), v2 = mul2(r, r);
        update(a.c, k, gv[x], pv[x], mv[2 * u + x], v2, rv[2 * u + x]);
      }
      now.p.set(u, pv);
      z.add(now.p.four(u), n - i - 4 * u);
    }
    // values behind the end are zeros: they neither raise a scale nor are stored
    float sm, sv;
    encode<false>(mv, now.m, sm);
    encode<true>(rv, now.v, sv);
    if (vec && i + kWide8 <= n) {
      now.p.store(p + i);
      now.m.store(m + i);
      now.v.store(v + i);
    } else {
      now.p.put(p + i, n - i);
      now.m.put(m + i, n - i);
      now.v.put(v + i, n - i);
    }
    if (threadIdx.x % 8 == 0 && i < n) {
      ms[i / kBlock] = sm;
      vs[i / kBlock] = sv;
    }
  }
  if (!z.all()) set_status(a.c.status, MC_STATUS_NONFINITE_UPDATE);
}

template <typename P, typename G, bool EIGHT, int N>
cudaError_t launch(const Tensor* t, int count, int steps, uint32_t chunks, const Coef& c, cudaStream_t s) {
  Launch<N> a;
  memcpy(a.t, t, (size_t)count * sizeof(Tensor));
  a.c = c;
  a.count = count;
  a.steps = steps;
  if constexpr (EIGHT) return launch_behind(adamw8_kernel<P, G, N>, chunks, kThreads, 0, s, a);
  else return launch_behind(adamw_kernel<P, G, N>, chunks, kThreads, 0, s, a);
}
// A launch's tensors travel among its parameters, at most 32,764 bytes of them:
// few where few do, since the driver copies them all.
constexpr int kFew = 16, kSome = 128, kMany = 504;
static_assert(sizeof(Launch<kMany>) <= 32764, "kernel parameters");
template <typename P, typename G, bool EIGHT>
cudaError_t launch_any(const Tensor* t, int count, int steps, uint32_t chunks, const Coef& c, cudaStream_t s) {
  if (count <= kFew) return launch<P, G, EIGHT, kFew>(t, count, steps, chunks, c, s);
  if (count <= kSome) return launch<P, G, EIGHT, kSome>(t, count, steps, chunks, c, s);
  return launch<P, G, EIGHT, kMany>(t, count, steps, chunks, c, s);
}

mc_status err(mc_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}

struct Span {
  uintptr_t lo, hi;
  bool out;
  int index;
  const char* name;
};

mc_status step(const mc_adamw_tensor* t, int32_t count, const mc_adamw_hparams* hp, const float* grad_scale, int32_t* status,
               cudaStream_t stream) {
  const char* me = "mc_adamw_step";
  if (count < 0 || (count > 0 && !t) || !hp) return err(MC_ERR_INVALID_ARG, "%s: need tensors and hyper-parameters", me);
  auto unit = [](double b) { return b >= 0.0 && b < 1.0; };
  if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay) || !std::isfinite(hp->eps) || hp->eps < 0.0)
    return err(MC_ERR_INVALID_ARG, "%s: lr, weight_decay and eps must be finite, eps >= 0", me);
  if (!unit(hp->beta1) || !unit(hp->beta2)) return err(MC_ERR_INVALID_ARG, "%s: beta1 and beta2 must be in [0, 1)", me);
  if (!hp->step_device && hp->step < 1) return err(MC_ERR_INVALID_ARG, "%s: step %lld, the first is 1", me, (long long)hp->step);
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (at(hp->step_device) % 8 || at(grad_scale) % 4 || at(status) % 4)
    return err(MC_ERR_INVALID_ARG, "%s: step_device, grad_scale or status is not aligned to its type", me);
  // memory by operand: a list's tensors often lie in their order
  std::vector<Span> spans[7];
  for (auto& x : spans) x.reserve((size_t)count + 1);
  auto span = [&](int kind, const char* name, int i, const void* p, int64_t bytes, bool out) {
    if (bytes > 0) spans[kind].push_back({at(p), at(p) + (uintptr_t)bytes, out, i, name});
  };
  // tensors of one set of types share a launch
  std::vector<Tensor> sorted[8];
  for (int i = 0; i < count; ++i) {
    const mc_adamw_tensor& a = t[i];
    if (a.n < 0 || a.n > (1ll << 40)) return err(MC_ERR_INVALID_ARG, "%s: tensor %d has %lld values", me, i, (long long)a.n);
    if ((a.p_dtype != MC_BF16 && a.p_dtype != MC_F32) || (a.g_dtype != MC_BF16 && a.g_dtype != MC_F32) ||
        (a.state_dtype != MC_F32 && a.state_dtype != MC_F8E4M3))
      return err(MC_ERR_INVALID_ARG, "%s: tensor %d has dtypes %d, %d, %d", me, i, a.p_dtype, a.g_dtype, a.state_dtype);
    if (a.n == 0) continue;
    const bool eight = a.state_dtype == MC_F8E4M3;
    if (eight && !(hp->beta1 <= MC_ADAMW_8BIT_BETA && hp->beta2 <= MC_ADAMW_8BIT_BETA))
      return err(MC_ERR_UNSUPPORTED, "%s: tensor %d: 8-bit states take betas up to %g, these are %g and %g", me, i, MC_ADAMW_8BIT_BETA,
                 hp->beta1, hp->beta2);
    const size_t ps = a.p_dtype == MC_BF16 ? 2 : 4, gs = a.g_dtype == MC_BF16 ? 2 : 4, ss = eight ? 1 : 4;
    if (!a.p || !a.g || !a.m || !a.v) return err(MC_ERR_INVALID_ARG, "%s: tensor %d: null pointer", me, i);
    if (eight != (a.m_scale != nullptr) || eight != (a.v_scale != nullptr))
      return err(MC_ERR_INVALID_ARG, "%s: tensor %d: scales go with 8-bit states", me, i);
    if (at(a.p) % ps || at(a.g) % gs || at(a.m) % ss || at(a.v) % ss || at(a.m_scale) % 4 || at(a.v_scale) % 4)
      return err(MC_ERR_INVALID_ARG, "%s: tensor %d: a pointer is not aligned to its type", me, i);
    const int64_t scales = eight ? cdiv(a.n, kBlock) * 4 : 0;
    span(0, "p", i, a.p, a.n * ps, true);
    span(1, "g", i, a.g, a.n * gs, false);
    span(2, "m", i, a.m, a.n * ss, true);
    span(3, "v", i, a.v, a.n * ss, true);
    span(4, "m_scale", i, a.m_scale, scales, true);
    span(5, "v_scale", i, a.v_scale, scales, true);
    const bool vec = eight ? at(a.p) % 32 == 0 && at(a.g) % 32 == 0 && at(a.m) % 16 == 0 && at(a.v) % 16 == 0
                           : at(a.p) % (4 * ps) == 0 && at(a.g) % (4 * gs) == 0 && at(a.m) % 16 == 0 && at(a.v) % 16 == 0;
    sorted[(a.p_dtype == MC_BF16) + 2 * (a.g_dtype == MC_BF16) + 4 * eight].push_back(
        {a.p, a.g, a.m, a.v, a.m_scale, a.v_scale, a.n, 0u, vec ? 1u : 0u});
  }
  span(6, "step_device", -1, hp->step_device, hp->step_device ? 8 : 0, false);
  span(6, "grad_scale", -1, grad_scale, grad_scale ? 4 : 0, false);
  span(6, "status", -1, status, status ? 4 : 0, true);
  // what is written shares memory with nothing
  auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  std::vector<Span> every;
  every.reserve(6 * (size_t)count + 3);
  for (auto& x : spans) {
    if (!std::is_sorted(x.begin(), x.end(), before)) std::sort(x.begin(), x.end(), before);
    const auto middle = (ptrdiff_t)every.size();
    every.insert(every.end(), x.begin(), x.end());
    if (middle > 0 && !x.empty() && before(x.front(), every[(size_t)middle - 1]))
      std::inplace_merge(every.begin(), every.begin() + middle, every.end(), before);
  }
  const Span *far = nullptr, *far_out = nullptr;        // of those before, the one (written) that reaches furthest
  for (const Span& s : every) {
    const Span* with = s.out ? far : far_out;
    if (with && with->hi > s.lo)
      return err(MC_ERR_INVALID_ARG, "%s: %s of tensor %d overlaps %s of tensor %d", me, s.name, s.index, with->name, with->index);
    if (!far || s.hi > far->hi) far = &s;
    if (s.out && (!far_out || s.hi > far_out->hi)) far_out = &s;
  }
  Coef c;
  memset(&c, 0, sizeof c);
  c.b1 = (float)hp->beta1;
  c.c1 = (float)(1.0 - hp->beta1);
  c.b2 = (float)hp->beta2;
  c.c2 = (float)(1.0 - hp->beta2);
  c.one = 1.f;
  c.lr = (float)hp->lr;
  c.wd = (float)hp->weight_decay;
  c.eps = (float)hp->eps;
  // log beta, of 0 too: at -200 and below a power is 0 in fp32
  auto parts = [](double beta, float (&to)[2]) {
    const double l = std::max(std::log(beta), -200.0);
    to[0] = (float)l;
    to[1] = (float)(l - (double)to[0]);
  };
  parts(hp->beta1, c.l1);
  parts(hp->beta2, c.l2);
  c.step = reinterpret_cast<const long long*>(hp->step_device);
  if (!c.step) {
    c.i1 = (float)(-1.0 / std::expm1((double)hp->step * std::log(hp->beta1)));         // log 0 = -inf: 1
    c.i2 = (float)(1.0 / std::sqrt(-std::expm1((double)hp->step * std::log(hp->beta2))));
  }
  c.grad_scale = grad_scale;
  c.status = status;
  using Any = cudaError_t (*)(const Tensor*, int, int, uint32_t, const Coef&, cudaStream_t);
  using B = __nv_bfloat16;
  static const Any by_types[8] = {launch_any<float, float, false>, launch_any<B, float, false>, launch_any<float, B, false>,
                                  launch_any<B, B, false>,         launch_any<float, float, true>, launch_any<B, float, true>,
                                  launch_any<float, B, true>,      launch_any<B, B, true>};
  for (int k = 0; k < 8; ++k) {
    std::vector<Tensor>& own = sorted[k];
    long long values = 0;
    for (const Tensor& x : own) values += x.n;
    const int set = kThreads * (k < 4 ? kWide : kWide8);
    int steps = k < 4 ? kSteps : kSteps8;
    while (steps > (k < 4 ? kAhead : 1) && values < (long long)sm_count() * kPerSm * steps * set) steps /= 2;
    for (size_t i = 0; i < own.size();) {
      uint32_t chunks = 0;
      size_t j = i;
      for (; j < own.size() && j - i < kMany; ++j) {
        const long long more = cdiv(own[j].n, steps * set);
        if (chunks + more > 0x7fffffffll) break;        // 2^40 values are at most 2^28 chunks: the first always fits
        own[j].begin = chunks;
        chunks += (uint32_t)more;
      }
      const cudaError_t e = by_types[k](own.data() + i, (int)(j - i), steps, chunks, c, stream);
      if (e != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(e));
      i = j;
    }
  }
  return record_error(MC_OK, "");
}

}  // namespace aw
}  // namespace
}  // namespace mc

extern "C" mc_status mc_adamw_step(const mc_adamw_tensor* t, int32_t count, const mc_adamw_hparams* hp,
                                   const float* grad_scale, int32_t* status, mc_stream_t stream) {
  try {
    return mc::aw::step(t, count, hp, grad_scale, status, (cudaStream_t)stream);
  } catch (const std::exception& e) {      // memory of the host's lists
    return mc::aw::err(MC_ERR_INVALID_ARG, "mc_adamw_step: %s", e.what());
  }
}
