// Setup (untimed): the query/key features of an attention layer on the
// library's own kernels, so that S_max and its re-measurement after a clip run
// entirely on the library.  [K2-internals] "MLA 的特殊处理": the query splits
// into a per-head part q^C and a rotary part q^R taken from the compressed
// query latent; the keys into k^C (per head, from the compressed key/value
// latent) and one rotary k^R shared by every head.  MHA: Q = X W_q^T,
// K = X W_k^T ([K2-notes] 3.2).
//
//   mc_matmul    D = A B^T: bf16 on the Newton-Schulz GEMM core (tcgen05 CTA
//                pairs, one bf16 plane, fp32 accumulation); fp32 on the
//                CUDA-core GEMM with compensated sums.
//   mc_rms_norm  y = x / sqrt(mean(x^2) + eps) per row (weightless RMSNorm of
//                the latents), fp32 arithmetic.
//   mc_rope      rotary embedding on interleaved pairs at positions 0..S-1,
//                angles s * theta^(-2k/d) and their cosines and sines in fp64.
//   mc_rope_backward  its gradient: the transposed rotation.
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

template <typename T>
__device__ inline float ldv(const T* p);
template <>
__device__ inline float ldv<float>(const float* p) { return *p; }
template <>
__device__ inline float ldv<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <typename T>
__device__ inline void stv(T* p, float v);
template <>
__device__ inline void stv<float>(float* p, float v) { *p = v; }
template <>
__device__ inline void stv<__nv_bfloat16>(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One warp per row: the mean of the squares over `cols` values in fp32, then
// every value divided by sqrt(mean + eps).  In place when y == x (each value
// is read and then written by the same lane).
template <typename T>
__global__ void rms_rows_kernel(const T* x, long long ldx, T* y, long long ldy, long long rows, int cols,
                                float eps) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  for (long long r = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += warps) {
    const T* xr = x + r * ldx;
    T* yr = y + r * ldy;
    float s = 0.f;
    for (int c = lane; c < cols; c += 32) {
      const float v = ldv(xr + c);
      s = fmaf(v, v, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float inv = 1.f / sqrtf(s / (float)cols + eps);
    for (int c = lane; c < cols; c += 32) stv(yr + c, ldv(xr + c) * inv);
  }
}

// One (b, s) position per iteration of a block: the d/2 cosines and sines of
// position s go to shared memory (fp64 angle, rounded to fp32), then every
// head's pairs (x[2k], x[2k+1]) rotate by them, in place.
template <typename T>
__global__ void rope_kernel(T* x, int B, int S, int nh, int d, long long sb, long long ss, long long sh,
                            double theta) {
  extern __shared__ float cs[];          // [d/2] cosines, then [d/2] sines
  const int half = d / 2;
  const long long rows = (long long)B * S;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const int b = (int)(row / S), s = (int)(row % S);
    __syncthreads();
    for (int k = threadIdx.x; k < half; k += blockDim.x) {
      const double ang = (double)s * pow(theta, -2.0 * (double)k / (double)d);
      double sn, cn;
      sincos(ang, &sn, &cn);
      cs[k] = (float)cn;
      cs[half + k] = (float)sn;
    }
    __syncthreads();
    T* xr = x + (long long)b * sb + (long long)s * ss;
    for (int i = threadIdx.x; i < nh * half; i += blockDim.x) {
      const int h = i / half, k = i - h * half;
      T* p = xr + (long long)h * sh + 2 * k;
      const float x0 = ldv(p), x1 = ldv(p + 1), c = cs[k], sn = cs[half + k];
      stv(p, x0 * c - x1 * sn);
      stv(p + 1, x0 * sn + x1 * c);
    }
  }
}

// Gradient of the rotary embedding: the transposed rotation of each pair, from
// dy to dx (which may be dy).  A thread owns V pairs (16 bytes) of one position
// and walks over a group of heads, eight loads in flight, so it needs its sines
// and cosines once.  A pair's turns per position are a sum of two fp32 (from fp64,
// once per block, under the first loads), and the turns at a position are reduced
// to at most half a turn exactly: s hi and its rounding error, plus s lo.  So the
// fp32 sine and cosine are good to 2^-22 absolute at any angle up to 2^24 (two
// fp32 hold 2^-48 of the turn per position; larger ones are refused) without fp64
// arithmetic per position (this part runs it at a fraction of fp32's rate).  Bound
// by memory and its latency: [1, 4096, 64, 64] bf16, 67 MB, takes 11.6 us (5.8
// TB/s); a table of sines per block in shared memory, as in the forward, cost two
// barriers per few positions (18 us).
struct RopeBack {
  const void* dy; void* dx;
  long long yb, ys, yh, xb, xs, xh;
  int S, nh, d;
  int heads;                             // per thread
  int total;                             // threads that have work
  double step;                           // log2(theta) * 2 / d
  FastDiv div_nv, div_s, div_groups;
};
constexpr int kRopeFlight = 8;
// (a, b) -> (a c + b s, b c - a s)
__device__ inline void turn_back(float& a, float& b, float c, float s) {
  untwo(fma2(two(b, a), two(s, -s), mul2(two(a, b), two(c, c))), a, b);
}
// V pairs of one head and position: one 16-byte access, or two single values.
template <typename T, int V>
struct PairsOf;
template <>
struct PairsOf<__nv_bfloat16, 4> {
  uint32_t w[4];
  __device__ void load(const __nv_bfloat16* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ void turn_back(const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xffff0000u);
      mc::turn_back(a, b, c[k], s[k]);
      const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
      w[k] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};
template <>
struct PairsOf<float, 2> {
  float4 w;
  __device__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ void turn_back(const float (&c)[2], const float (&s)[2]) {
    mc::turn_back(w.x, w.y, c[0], s[0]);
    mc::turn_back(w.z, w.w, c[1], s[1]);
  }
};
template <typename T>
struct PairsOf<T, 1> {
  T a, b;
  __device__ void load(const T* p) { a = p[0]; b = p[1]; }
  __device__ void store(T* p) const { p[0] = a; p[1] = b; }
  __device__ void turn_back(const float (&c)[1], const float (&s)[1]) {
    float x = ldv(&a), y = ldv(&b);
    mc::turn_back(x, y, c[0], s[0]);
    stv(&a, x);
    stv(&b, y);
  }
};

template <typename T, int V>
__global__ void __launch_bounds__(256, 4) rope_back_kernel(const __grid_constant__ RopeBack p) {
  extern __shared__ float2 turns[];      // [d/2] (hi, lo) turns per position
  await_previous();
  release_next();
  const int half = p.d / 2, nv = half / V;
  const int t = (int)(blockIdx.x * 256 + threadIdx.x);
  const int r0 = (int)fastdiv(t, p.div_nv), c = t - r0 * nv;
  const int r1 = (int)fastdiv(r0, p.div_s), s = r0 - r1 * p.S;
  const int b = (int)fastdiv(r1, p.div_groups);
  const int groups = (p.nh + p.heads - 1) / p.heads;
  const int h0 = (r1 - b * groups) * p.heads, h1 = t < p.total ? min(p.nh, h0 + p.heads) : h0;
  const T* src = static_cast<const T*>(p.dy) + b * p.yb + s * p.ys + 2 * V * c;
  T* dst = static_cast<T*>(p.dx) + b * p.xb + s * p.xs + 2 * V * c;
  PairsOf<T, V> q[kRopeFlight];
  // heads h .. h + 7 of the group (those that it has)
  auto load = [&](int h) {
    const T* from = src + h * p.yh;
#pragma unroll
    for (int n = 0; n < kRopeFlight; ++n, from += p.yh)
      if (h + n < h1) q[n].load(from);
  };
  load(h0);
  for (int k = threadIdx.x; k < half; k += 256) {
    const double x = exp2(-p.step * k) * 0.15915494309189535;
    const float hi = (float)x;
    turns[k] = make_float2(hi, (float)(x - hi));
  }
  __syncthreads();
  float cn[V], sn[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float2 f = turns[V * c + k];
    const float at = (float)s, x = at * f.x, e = fmaf(at, f.x, -x);
    sincospif(2.f * ((x - rintf(x)) + fmaf(at, f.y, e)), &sn[k], &cn[k]);
  }
  for (int h = h0; h < h1; h += kRopeFlight) {
    if (h > h0) load(h);
    T* to = dst + h * p.xh;
#pragma unroll
    for (int n = 0; n < kRopeFlight; ++n, to += p.xh)
      if (h + n < h1) {
        q[n].turn_back(cn, sn);
        q[n].store(to);
      }
  }
}

template <typename T, int V>
cudaError_t launch_rope_back(RopeBack p, int B, cudaStream_t s) {
  // heads are split over threads as long as four blocks per SM, which are
  // resident at once, take them
  const int nv = p.d / 2 / V;
  const long long at = (long long)B * p.S * nv, most = 4ll * 256 * sm_count() / at;
  const int ways = (int)(most < 1 ? 1 : most > p.nh ? p.nh : most);
  p.heads = (p.nh + ways - 1) / ways;
  const int groups = (p.nh + p.heads - 1) / p.heads;
  p.total = (int)(at * groups);          // below 2^31: at is checked, and groups > 1 stays within four blocks per SM
  p.div_nv = make_fastdiv((uint32_t)nv);
  p.div_s = make_fastdiv((uint32_t)p.S);
  p.div_groups = make_fastdiv((uint32_t)groups);
  return launch_behind(rope_back_kernel<T, V>, (unsigned)cdiv(at * groups, 256), 256, (size_t)(p.d / 2) * 8, s, p);
}

mc_status err(mc_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}

mc_status done() { return record_error(MC_OK, ""); }

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t esize(int32_t dtype) { return dtype == MC_BF16 ? 2 : 4; }

}  // namespace
}  // namespace mc

using namespace mc;

extern "C" {

mc_status mc_matmul(const void* A, int64_t lda, const void* B, int64_t ldb, void* D, int64_t ldd,
                    int32_t M, int32_t N, int32_t K, int32_t dtype, void* scratch, int32_t* status,
                    mc_stream_t stream) {
  if (dtype != MC_BF16 && dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "mc_matmul: dtype %d", dtype);
  if (M < 0 || N < 0 || K < 1) return err(MC_ERR_INVALID_ARG, "mc_matmul: M %d, N %d, K %d", M, N, K);
  if (M == 0 || N == 0) return done();
  if (!A || !B || !D) return err(MC_ERR_INVALID_ARG, "mc_matmul: null operand");
  if (lda < K || ldb < K || ldd < N) return err(MC_ERR_INVALID_ARG, "mc_matmul: pitch below the row length");
  const size_t es = esize(dtype);
  if (!al16(A) || !al16(B) || !al16(D) || (lda * es) % 16 || (ldb * es) % 16 || (ldd * es) % 16)
    return err(MC_ERR_INVALID_ARG, "mc_matmul: pointers and row pitches must be 16-byte aligned");
  if (dtype == MC_BF16 && (!scratch || !al16(scratch)))
    return err(MC_ERR_INVALID_ARG, "mc_matmul: bf16 needs a 16-byte aligned device scratch of >= 16 bytes");
  GemmParams gp;
  memset(&gp, 0, sizeof gp);
  gp.xmode = dtype == MC_BF16 ? kXBf16 : kXF32;
  gp.status = status;
  gp.ngroups = 1;
  gp.terms = 1;
  gp.fmt = kFmtBf16;
  gp.alpha = 1.f;
  GemmGroup& G = gp.g[0];
  G.M = M; G.N = N; G.K = K; G.batch = 1;
  G.a_hi = A; G.lda = lda; G.a_bstride = (long long)M * lda;
  G.b_hi = B; G.ldb = ldb; G.b_bstride = (long long)N * ldb;
  G.d_hi = D; G.ldd = ldd; G.d_bstride = (long long)M * ldd;
  const int tm = dtype == MC_BF16 ? kTcTileM : 64, tn = dtype == MC_BF16 ? kTcTileN : 64;
  G.tiles_m = (int)cdiv(M, tm);
  G.tiles_n = (int)cdiv(N, tn);
  G.tiles_per_item = G.tiles_m * G.tiles_n;
  gp.total_tiles = G.tiles_per_item;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == MC_BF16) {
    e = cudaMemsetAsync(scratch, 0, sizeof(int), s);          // the launch's tile counter
    if (e != cudaSuccess) return err(MC_ERR_CUDA, "mc_matmul: %s", cudaGetErrorString(e));
    gp.sched = static_cast<int*>(scratch);
    char msg[256] = {0};
    e = launch_ns_gemm_tc(gp, nullptr, s, msg, sizeof msg);
    if (e != cudaSuccess && msg[0]) return err(MC_ERR_CUDA, "mc_matmul: tensor-core GEMM: %s", msg);
  } else {
    e = launch_ns_gemm_f32(gp, s);
  }
  if (e != cudaSuccess) return err(MC_ERR_CUDA, "mc_matmul: %s", cudaGetErrorString(e));
  return done();
}

mc_status mc_rms_norm(const void* x, int64_t ldx, void* y, int64_t ldy, int64_t rows, int32_t cols,
                      int32_t dtype, float eps, mc_stream_t stream) {
  if (dtype != MC_BF16 && dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "mc_rms_norm: dtype %d", dtype);
  if (rows < 0 || cols < 1 || ldx < cols || ldy < cols)
    return err(MC_ERR_INVALID_ARG, "mc_rms_norm: rows %lld, cols %d, pitches %lld / %lld", (long long)rows,
               cols, (long long)ldx, (long long)ldy);
  if (!(eps >= 0.f)) return err(MC_ERR_INVALID_ARG, "mc_rms_norm: eps must be >= 0");
  if (rows == 0) return done();
  if (!x || !y) return err(MC_ERR_INVALID_ARG, "mc_rms_norm: null pointer");
  const int threads = 256, rows_per_block = threads / 32;
  const long long want = (rows + rows_per_block - 1) / rows_per_block;
  const int grid = (int)(want < (long long)sm_count() * 8 ? want : (long long)sm_count() * 8);
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MC_BF16)
    rms_rows_kernel<__nv_bfloat16><<<grid, threads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), ldx,
                                                            static_cast<__nv_bfloat16*>(y), ldy, rows, cols, eps);
  else
    rms_rows_kernel<float><<<grid, threads, 0, s>>>(static_cast<const float*>(x), ldx, static_cast<float*>(y),
                                                    ldy, rows, cols, eps);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return err(MC_ERR_CUDA, "mc_rms_norm: %s", cudaGetErrorString(e));
  return done();
}

mc_status mc_rope(void* x, int32_t B, int32_t S, int32_t nh, int32_t d, int64_t sb, int64_t ss, int64_t sh,
                  int32_t dtype, double theta, mc_stream_t stream) {
  if (dtype != MC_BF16 && dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "mc_rope: dtype %d", dtype);
  if (B < 0 || S < 0 || nh < 1 || d < 2 || (d & 1) || d > 4096)
    return err(MC_ERR_INVALID_ARG, "mc_rope: B %d, S %d, heads %d, d %d (d even, 2..4096)", B, S, nh, d);
  if (!(theta > 0.0)) return err(MC_ERR_INVALID_ARG, "mc_rope: theta must be > 0");
  if ((long long)B * S == 0) return done();
  if (!x) return err(MC_ERR_INVALID_ARG, "mc_rope: null pointer");
  const long long rows = (long long)B * S;
  const int grid = (int)(rows < (long long)sm_count() * 8 ? rows : (long long)sm_count() * 8);
  const size_t smem = (size_t)d * sizeof(float);
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == MC_BF16)
    rope_kernel<__nv_bfloat16><<<grid, 256, smem, s>>>(static_cast<__nv_bfloat16*>(x), B, S, nh, d, sb, ss, sh,
                                                        theta);
  else
    rope_kernel<float><<<grid, 256, smem, s>>>(static_cast<float*>(x), B, S, nh, d, sb, ss, sh, theta);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return err(MC_ERR_CUDA, "mc_rope: %s", cudaGetErrorString(e));
  return done();
}

mc_status mc_rope_backward(const void* dy, int64_t yb, int64_t ys, int64_t yh, void* dx, int64_t xb, int64_t xs,
                           int64_t xh, int32_t B, int32_t S, int32_t nh, int32_t d, int32_t dtype, double theta,
                           mc_stream_t stream) {
  const char* me = "mc_rope_backward";
  if (dtype != MC_BF16 && dtype != MC_F32) return err(MC_ERR_INVALID_ARG, "%s: dtype %d", me, dtype);
  if (B < 0 || S < 0 || nh < 1 || d < 2 || (d & 1) || d > 4096)
    return err(MC_ERR_INVALID_ARG, "%s: B %d, S %d, heads %d, d %d (d even, 2..4096)", me, B, S, nh, d);
  if (!(theta > 0.0) || !std::isfinite(theta)) return err(MC_ERR_INVALID_ARG, "%s: theta must be finite and > 0", me);
  if ((long long)B * S == 0) return done();
  // positions are exact as fp32, and angles keep the accuracy of their two-fp32 turns
  if (S * (theta < 1.0 ? 1.0 / theta : 1.0) > 0x1p24)
    return err(MC_ERR_UNSUPPORTED, "%s: S %d, theta %g: angles beyond 2^24 are too large", me, S, theta);
  if (!dy || !dx) return err(MC_ERR_INVALID_ARG, "%s: null pointer", me);
  const size_t es = esize(dtype);
  if (reinterpret_cast<uintptr_t>(dy) % es || reinterpret_cast<uintptr_t>(dx) % es)
    return err(MC_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", me);
  const int64_t ext[3] = {B, S, nh}, sy[3] = {yb, ys, yh}, sx[3] = {xb, xs, xh};
  int64_t endy = d, endx = d;
  bool same = dy == dx, vec = d % (16 / es) == 0 && al16(dy) && al16(dx);
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;
    if (sy[i] < 0 || sx[i] < 0) return err(MC_ERR_INVALID_ARG, "%s: negative stride", me);
    endy += (ext[i] - 1) * sy[i];
    endx += (ext[i] - 1) * sx[i];
    same = same && sy[i] == sx[i];
    vec = vec && (sy[i] * es) % 16 == 0 && (sx[i] * es) % 16 == 0;
  }
  if (!distinct_addresses(sx, ext, 3, d)) return err(MC_ERR_INVALID_ARG, "%s: elements of dx share addresses", me);
  const uintptr_t py = reinterpret_cast<uintptr_t>(dy), px = reinterpret_cast<uintptr_t>(dx);
  if (!same && py < px + endx * es && px < py + endy * es)
    return err(MC_ERR_INVALID_ARG, "%s: dx overlaps dy without being dy", me);
  if ((long long)B * S > (1ll << 31) / (d / 2) / 2) return err(MC_ERR_UNSUPPORTED, "%s: B %d, S %d, d %d are too large", me, B, S, d);
  RopeBack p;
  memset(&p, 0, sizeof p);
  p.dy = dy; p.dx = dx;
  p.yb = yb; p.ys = ys; p.yh = yh;
  p.xb = xb; p.xs = xs; p.xh = xh;
  p.S = S; p.nh = nh; p.d = d;
  p.step = std::log2(theta) * 2.0 / d;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == MC_BF16) e = vec ? launch_rope_back<__nv_bfloat16, 4>(p, B, s) : launch_rope_back<__nv_bfloat16, 1>(p, B, s);
  else e = vec ? launch_rope_back<float, 2>(p, B, s) : launch_rope_back<float, 1>(p, B, s);
  if (e != cudaSuccess) return err(MC_ERR_CUDA, "%s: %s", me, cudaGetErrorString(e));
  return done();
}

}  // extern "C"
