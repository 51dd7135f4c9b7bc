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
// becomes zero (the least code is 2^-9): a forgotten v would divide its next
// gradient by eps alone.  The parameter's step takes m and v before their
// rounding.
//
// One pass over memory, 22 bytes a value with bf16 p and g and fp32 states, 10.1
// with 8-bit ones.  A block takes a chunk of one tensor and finds which by a
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
#include <type_traits>
#include <vector>

#include "../../include/muonclip.h"
#include "common.cuh"
#include "kernels.h"

namespace mc {
namespace {
namespace aw {

constexpr int kThreads = 256;
constexpr int kSets = 4;                          // groups of four values per thread and chunk
constexpr int kAhead = 2;                         // sets in flight
constexpr int kChunk = kThreads * 4 * kSets;      // values per block
constexpr int kBlock = MC_ADAMW_BLOCK;            // values per scale: a warp's 32 x 4
static_assert(kBlock == 128 && kChunk % kBlock == 0, "a warp holds whole blocks");
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
  uint32_t vec;                                   // every operand aligned to four of its values
};
struct Coef {
  float b1, c1, b2, c2;                           // beta1, 1 - beta1, beta2, 1 - beta2
  float lr, wd, eps;
  float i1, i2;                                   // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double l1, l2;                                  // log beta1, log beta2 (for a step on the device)
  const long long* step;                          // or null
  const float* grad_scale;                        // or null
  int32_t* status;
};
template <int N>
struct Launch {
  Tensor t[N];
  Coef c;
  int count;
};

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
  __device__ void get(float (&x)[4]) const { x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w; }
  __device__ void set(const float (&x)[4]) { w = make_float4(x[0], x[1], x[2], x[3]); }
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
  __device__ void get(float (&x)[4]) const {
    x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  __device__ void set(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ void put(__nv_bfloat16* p, int n) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = __ushort_as_bfloat16((unsigned short)((i < 2 ? w.x : w.y) >> (16 * (i & 1))));
  }
};
// Four e4m3 codes.
struct Codes {
  uint32_t w;
  __device__ void load(const uint8_t* p) { w = *reinterpret_cast<const uint32_t*>(p); }
  __device__ void part(const uint8_t* p, int n) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) w |= (uint32_t)p[i] << (8 * i);
  }
  __device__ void get(float (&x)[4]) const {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 u = __half22float2(__half2(a)), v = __half22float2(__half2(b));
    x[0] = u.x; x[1] = u.y; x[2] = v.x; x[3] = v.y;
  }
  __device__ void set(const float (&x)[4]) {
    w = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3) |
        (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3) << 16;
  }
  __device__ void store(uint8_t* p) const { *reinterpret_cast<uint32_t*>(p) = w; }
  __device__ void put(uint8_t* p, int n) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint8_t)(w >> (8 * i));
  }
};

// max|x| over the warp, NaN if one is (as unsigned integers, non-negative values
// keep their order and every NaN lies above them).
__device__ inline float warp_max(const float (&x)[4]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = max(a, __float_as_uint(fabsf(x[i])));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, a));
}
// Codes of 128 values of a warp, and their scale.  Every operation is one rounding
// of its operands' (no contraction), so equal states give equal codes wherever
// they are computed so.
template <bool ROOT>
__device__ inline void encode(float (&x)[4], Codes& code, float& scale) {
  const float q = __fmul_rn(warp_max(x), 1.f / 448.f);
  scale = q < kScaleMin ? kScaleMin : q;          // NaN stays NaN, as fmaxf would not let it
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = __fmul_rn(x[i], inv);
    x[i] = ROOT && y > 0.f && y < kLeast ? kLeast : y;
  }
  code.set(x);
}

// A thread's four values of one set, as they lie in memory.
template <typename P, typename G, bool EIGHT>
struct Raw {
  Four<P> p;
  Four<G> g;
  typename std::conditional<EIGHT, Codes, Four<float>>::type m, v;
  float ms, vs;
};

template <typename P, typename G, bool EIGHT, int N>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Launch<N> a) {
  await_previous();
  release_next();
  // the last tensor whose first chunk is at or before this block
  int lo = 0;
#pragma unroll
  for (int step = N > 256 ? 256 : N / 2; step > 0; step >>= 1)      // N is 504 or a power of two
    if (lo + step < a.count && a.t[lo + step].begin <= blockIdx.x) lo += step;
  const Tensor& t = a.t[lo];
  const long long first = (long long)(blockIdx.x - t.begin) * kChunk;
  using S = typename std::conditional<EIGHT, uint8_t, float>::type;
  P* p = static_cast<P*>(t.p) + first;
  const G* g = static_cast<const G*>(t.g) + first;
  S *m = static_cast<S*>(t.m) + first, *v = static_cast<S*>(t.v) + first;
  float *ms = EIGHT ? t.ms + first / kBlock : nullptr, *vs = EIGHT ? t.vs + first / kBlock : nullptr;
  const int n = (int)min(t.n - first, (long long)kChunk);             // values of this chunk
  const bool vec = t.vec;
  float i1 = a.c.i1, i2 = a.c.i2;
  if (a.c.step) {
    const double at = (double)max(*a.c.step, 1ll);
    i1 = (float)(-1.0 / expm1(at * a.c.l1));
    i2 = (float)(1.0 / sqrt(-expm1(at * a.c.l2)));
  }
  const float gs = a.c.grad_scale ? *a.c.grad_scale : 1.f;
  float z = 0.f;                                   // zero, or NaN once a new p is not finite
  Raw<P, G, EIGHT> raw[kAhead];
  auto load = [&](int s, Raw<P, G, EIGHT>& r) {
    const int i = s * (kThreads * 4) + threadIdx.x * 4;
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
    if (EIGHT && (i & ~(kBlock - 1)) < n) {
      r.ms = ms[i / kBlock];
      r.vs = vs[i / kBlock];
    }
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) load(s, raw[s]);
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int i = s * (kThreads * 4) + threadIdx.x * 4;
    if ((i & ~(kBlock - 1)) >= n) break;           // the whole warp is behind the end
    const Raw<P, G, EIGHT> now = raw[s % kAhead];
    if (s + kAhead < kSets) load(s + kAhead, raw[s % kAhead]);
    float pv[4], gv[4], mv[4], vv[4], r[4];
    now.p.get(pv);
    now.g.get(gv);
    now.m.get(mv);
    now.v.get(vv);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (EIGHT) {
        mv[x] = __fmul_rn(mv[x], now.ms);
        vv[x] = __fmul_rn(vv[x], now.vs);
        vv[x] = __fmul_rn(vv[x], vv[x]);
      }
      const float gr = gv[x] * gs;
      mv[x] = __fadd_rn(__fmul_rn(mv[x], a.c.b1), __fmul_rn(gr, a.c.c1));
      vv[x] = __fadd_rn(__fmul_rn(vv[x], a.c.b2), __fmul_rn(__fmul_rn(gr, gr), a.c.c2));
      r[x] = __fsqrt_rn(vv[x]);
      // the quotient is of the order of 1 and moves p by lr of itself: an ulp or two of
      // it are nothing beside p's own rounding
      const float u = __fdividef(mv[x] * i1, fmaf(r[x], i2, a.c.eps));
      pv[x] = fmaf(-a.c.lr, fmaf(a.c.wd, pv[x], u), pv[x]);
    }
    Four<P> out;
    out.set(pv);
#pragma unroll
    for (int x = 0; x < 4; ++x) z = i + x < n ? fmaf(pv[x], 0.f, z) : z;
    if (vec && i + 4 <= n) out.store(p + i); else out.put(p + i, n - i);
    // lanes behind the end hold zeros: they neither raise a scale nor are stored
    typename std::conditional<EIGHT, Codes, Four<float>>::type cm, cv;
    if constexpr (EIGHT) {
      float sm, sv;
      encode<false>(mv, cm, sm);
      encode<true>(r, cv, sv);
      if ((threadIdx.x & 31) == 0) {
        ms[i / kBlock] = sm;
        vs[i / kBlock] = sv;
      }
    } else {
      cm.set(mv);
      cv.set(vv);
    }
    if (vec && i + 4 <= n) {
      cm.store(m + i);
      cv.store(v + i);
    } else {
      cm.put(m + i, n - i);
      cv.put(v + i, n - i);
    }
  }
  if (z != 0.f) set_status(a.c.status, MC_STATUS_NONFINITE_UPDATE);
}

template <typename P, typename G, bool EIGHT, int N>
cudaError_t launch(const Tensor* t, int count, uint32_t chunks, const Coef& c, cudaStream_t s) {
  Launch<N> a;
  memcpy(a.t, t, (size_t)count * sizeof(Tensor));
  a.c = c;
  a.count = count;
  return launch_behind(adamw_kernel<P, G, EIGHT, N>, chunks, kThreads, 0, s, a);
}
// A launch's tensors travel among its parameters, at most 32,764 bytes of them:
// few where few do, since the driver copies them all.
constexpr int kFew = 16, kSome = 128, kMany = 504;
static_assert(sizeof(Launch<kMany>) <= 32764, "kernel parameters");
template <typename P, typename G, bool EIGHT>
cudaError_t launch_any(const Tensor* t, int count, uint32_t chunks, const Coef& c, cudaStream_t s) {
  if (count <= kFew) return launch<P, G, EIGHT, kFew>(t, count, chunks, c, s);
  if (count <= kSome) return launch<P, G, EIGHT, kSome>(t, count, chunks, c, s);
  return launch<P, G, EIGHT, kMany>(t, count, chunks, c, s);
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
  std::vector<Span> spans;
  spans.reserve(6 * (size_t)count + 3);
  auto span = [&](const char* name, int i, const void* p, int64_t bytes, bool out) {
    if (bytes > 0) spans.push_back({at(p), at(p) + (uintptr_t)bytes, out, i, name});
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
    const size_t ps = a.p_dtype == MC_BF16 ? 2 : 4, gs = a.g_dtype == MC_BF16 ? 2 : 4, ss = eight ? 1 : 4;
    if (!a.p || !a.g || !a.m || !a.v) return err(MC_ERR_INVALID_ARG, "%s: tensor %d: null pointer", me, i);
    if (eight != (a.m_scale != nullptr) || eight != (a.v_scale != nullptr))
      return err(MC_ERR_INVALID_ARG, "%s: tensor %d: scales go with 8-bit states", me, i);
    if (at(a.p) % ps || at(a.g) % gs || at(a.m) % ss || at(a.v) % ss || at(a.m_scale) % 4 || at(a.v_scale) % 4)
      return err(MC_ERR_INVALID_ARG, "%s: tensor %d: a pointer is not aligned to its type", me, i);
    const int64_t scales = eight ? cdiv(a.n, kBlock) * 4 : 0;
    span("p", i, a.p, a.n * ps, true);
    span("g", i, a.g, a.n * gs, false);
    span("m", i, a.m, a.n * ss, true);
    span("v", i, a.v, a.n * ss, true);
    span("m_scale", i, a.m_scale, scales, true);
    span("v_scale", i, a.v_scale, scales, true);
    const bool vec = at(a.p) % (4 * ps) == 0 && at(a.g) % (4 * gs) == 0 && at(a.m) % (4 * ss) == 0 && at(a.v) % (4 * ss) == 0;
    sorted[(a.p_dtype == MC_BF16) + 2 * (a.g_dtype == MC_BF16) + 4 * eight].push_back(
        {a.p, a.g, a.m, a.v, a.m_scale, a.v_scale, a.n, 0u, vec ? 1u : 0u});
  }
  span("step_device", -1, hp->step_device, hp->step_device ? 8 : 0, false);
  span("grad_scale", -1, grad_scale, grad_scale ? 4 : 0, false);
  span("status", -1, status, status ? 4 : 0, true);
  // what is written shares memory with nothing
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  const Span *far = nullptr, *far_out = nullptr;        // of those before, the one (written) that reaches furthest
  for (const Span& s : spans) {
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
  c.lr = (float)hp->lr;
  c.wd = (float)hp->weight_decay;
  c.eps = (float)hp->eps;
  c.l1 = std::log(hp->beta1);                           // -inf for 0: expm1 of it is -1
  c.l2 = std::log(hp->beta2);
  c.step = reinterpret_cast<const long long*>(hp->step_device);
  if (!c.step) {
    c.i1 = (float)(-1.0 / std::expm1((double)hp->step * c.l1));
    c.i2 = (float)(1.0 / std::sqrt(-std::expm1((double)hp->step * c.l2)));
  }
  c.grad_scale = grad_scale;
  c.status = status;
  using Any = cudaError_t (*)(const Tensor*, int, uint32_t, const Coef&, cudaStream_t);
  using B = __nv_bfloat16;
  static const Any by_types[8] = {launch_any<float, float, false>, launch_any<B, float, false>, launch_any<float, B, false>,
                                  launch_any<B, B, false>,         launch_any<float, float, true>, launch_any<B, float, true>,
                                  launch_any<float, B, true>,      launch_any<B, B, true>};
  for (int k = 0; k < 8; ++k) {
    std::vector<Tensor>& own = sorted[k];
    for (size_t i = 0; i < own.size();) {
      uint32_t chunks = 0;
      size_t j = i;
      for (; j < own.size() && j - i < kMany; ++j) {
        const long long more = cdiv(own[j].n, kChunk);
        if (chunks + more > 0x7fffffffll) break;        // 2^40 values are 2^28 chunks: the first always fits
        own[j].begin = chunks;
        chunks += (uint32_t)more;
      }
      const cudaError_t e = by_types[k](own.data() + i, (int)(j - i), chunks, c, stream);
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
