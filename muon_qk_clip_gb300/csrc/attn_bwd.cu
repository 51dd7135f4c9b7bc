// Attention backward that recomputes the probabilities ([K2-internals]
// "核心数学": O^h = softmax(scale * Q^h K^h^T) V^h), per (batch, head):
//
//   p_ij  = exp(scale q_i . k_j - lse_i)      (0 above the diagonal when causal)
//   delta_i = do_i . o_i
//   dv_j  = sum_i p_ij do_i
//   ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i  = scale sum_j ds_ij k_j
//   dk_j  = scale sum_i ds_ij q_i             (its shared rotary columns summed over the heads)
//
// Three launches on the caller's stream (two without a shared key; sequences of at
// most 16 positions have one kernel for the first two), no atomics on results, so
// equal inputs give equal bits:
//   rows_kernel     delta and -lse log2(e) of every row, padded to whole tiles
//   bwd_kernel      dkv_pass: an item is 128 keys, loop over query tiles:
//                   S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q;
//                   then dq_pass: 128 queries, loop over key tiles: S = Q K^T,
//                   dP = dO V^T, dQ += dS K
//   shared_kernel   the shared key's gradient, summed over the heads in order
// Two passes recompute S and dP (7 products for the 5 that the formulas need),
// but dQ never leaves the chip as partial sums: one pass would add a 128 x D
// fp32 tile to global memory per tile pair, in an order that changes the bits.
//
// Packed sequences with grouped heads (attn_packed.cu) take the same passes: an item
// is then a block of one sequence, from the plan's list, the dK / dV pass goes over
// the query tiles of every head of the key head's group, and every tile is bounded by
// its sequence.  With few blocks of keys an item takes a part of these query tiles, and
// a launch of its own (join_kernel) adds the parts' dK and dV up.  16384 tokens in eight
// documents, 32 / 8 heads of 128: 890 us at first and 1010 in a long run of calls, under
// the power limit, 1.07 and 0.94 PFLOP/s of the five products (of the seven that the passes
// compute 1.50 and 1.32); rows_kernel takes 46 of them, at 6 TB/s.
//
// P and dS go from the compute warps to the tensor core through tensor memory
// (the A operand of dV, dK and dQ), written over the columns of the S / dP that
// they came from, rounded to bf16 like every operand; sums are fp32.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "fastdiv.cuh"
#include "kernels.h"
#include "packed.cuh"

namespace mc {
namespace {
namespace ab {
using namespace attn;

constexpr int BM = 128;                  // rows of a work item: keys (dkv) or queries (dq)
// Warps: 0 producer, 1 MMA issuer, 2 and 3 idle (packed: rows of no sequence), 4..7 output, 8..15 compute (a
// warp reads the tensor-memory lanes of its index mod 4).  The launch's 128
// registers a thread are dealt out again per group of four warps: the sum over
// the groups, 88 + 72 + 176 + 176, is the launch's 4 x 128.
constexpr int kThreads = 512;
constexpr int kRegsIssue = 88, kRegsOutput = 72, kRegsCompute = 176;
constexpr int CH = BM * 128;             // one 128-row x 64-feature bf16 chunk (128-byte swizzle)
constexpr uint32_t kTmemCols = 512;
constexpr int kBarBytes = 512;           // mbarriers and item ring of one pass
constexpr float kLog2e = 1.4426950408889634f;

// Tiles of the dK / dV pass by the 64-wide chunks of q.k and d_v.  Tensor memory
// has 512 columns: dK and dV take 64 (nch + ncv), S^T and dP^T one per query of
// the tile, P^T (bf16 pairs) half of one.  Up to three chunks P^T has columns of
// its own beside 128-query tiles; with more it is written over S^T: 128 queries
// then still fit four chunks, 96 five.  (With P^T apart and 96 queries four chunks'
// pass took 385 us on dense_block, against 358: the smaller the tile, the more
// often the tensor core re-reads K and V from shared memory.)
__host__ __device__ constexpr bool p_apart(int nch, int ncv) { return nch + ncv < 4; }
__host__ __device__ constexpr int query_tile(int nch, int ncv) { return nch + ncv > 4 ? 96 : 128; }
__host__ __device__ constexpr int query_stages(int nch, int ncv) { return p_apart(nch, ncv) ? 3 : 2; }
// Keys per tile of the dQ pass: tensor memory holds dQ (64 nch columns), Q and dO
// as operands (32 each per chunk), S and dP (a column per key) and dS (half of
// one).  With three chunks of q.k 96 keys fit when only two chunks of Q are there
// and dO is not: the rest is read from shared memory, and values have one stage.
// (64 keys with all of Q and dO in tensor memory: 1439 us for 32768 tokens instead
// of 1404, 841 for k2_mla_layer instead of 835; 96 keys with dS over dP, so that
// dP waits for dQ: 1414 and 842.)
__host__ __device__ constexpr int key_tile(int nch, int ncv) { return nch > 1 ? 96 : 128; }
__host__ __device__ constexpr int q_in_tmem(int nch) { return nch < 3 ? nch : 2; }
__host__ __device__ constexpr bool do_in_tmem(int nch) { return nch < 3; }
constexpr int kKeyStages = 3;            // key tiles of the dQ pass, and value tiles where they fit
__host__ __device__ constexpr int value_stages(int nch, int ncv) { return nch < 3 ? 3 : ncv < 2 ? 2 : 1; }

struct Maps {
  CUtensorMap q, k, ks, v, d_o;          // inputs: 64-feature chunks of a tile's rows
};

struct Geo {
  int nch, nck, ncv;    // 64-wide chunks of q.k, of its head-specific part, of d_v
  int nb;               // 128-row blocks per (b, h)
  int nt;               // dkv: query tiles per (b, h)
  int items;            // blocks in all, below 2^30 (checked on the host)
  int heads;            // B H
  int group;            // (b, h) pairs per group of the work order
  int full;             // items in whole groups
  long long sp;         // padded row length of nlse and delta
  FastDiv div_h, div_group_items, div_group, div_last;
  // packed sequences only
  int q_heads;          // per key head
  int parts;            // of a key block's query tiles, at most
  packed::Order order[2];          // of the dK / dV and the dQ pass
  const packed::Block* blocks;     // the plan's list, heaviest first, and its length
  const int* count;
  int fill;             // MC_FILL_* bits
};

// Work order.  Item x is one 128-row block of one (b, h).  Causal blocks differ
// in work by up to nb to 1, so the CTAs take items from a counter, in groups of
// about 512 blocks ((b, h) pairs that L2 can hold, more than the CTAs in flight),
// heaviest block first within a group: the last group's light blocks fill the
// end.  (Equal pairs of blocks dealt out in advance left CTAs idle for 4 % of the
// time with 64 heads of 32 blocks, for 19 % with 2 of 256 or 16 of 32.)
__device__ inline void item_at(const AttnBwdParams& p, const Geo& g, int x, bool heavy_last, int& b, int& h, int& blk) {
  const uint32_t grp = fastdiv((uint32_t)x, g.div_group_items);
  const uint32_t rem = (uint32_t)x - grp * (uint32_t)(g.group * g.nb);
  const bool last = x >= g.full;
  const uint32_t rank = fastdiv(rem, last ? g.div_last : g.div_group);
  const uint32_t n = last ? (uint32_t)(g.heads - (int)grp * g.group) : (uint32_t)g.group;
  const uint32_t bh = grp * (uint32_t)g.group + (rem - rank * n);
  b = (int)fastdiv(bh, g.div_h);
  h = (int)(bh - (uint32_t)b * (uint32_t)p.H);
  blk = heavy_last && p.causal ? g.nb - 1 - (int)rank : (int)rank;
}

// The items go from the producer, which takes them from the counter, to the
// other warps through a ring in shared memory.  The producer takes and publishes
// the next item before it loads the current one's last tile: late, so that no
// CTA holds an item that another could begin, and early enough that no warp
// waits for it.
constexpr int kRing = 4;
struct Ring {
  volatile int* slot;   // [kRing]
  uint64_t* full;       // [kRing] 1 arrival
  uint64_t* empty;      // [kRing] an arrival from each of the 13 other warps
};
__device__ inline bool ring_put(const Ring& r, uint32_t n, int x, volatile int* abort_flag) {
  const int s = n % kRing;
  if (!mbar_wait(&r.empty[s], ((n / kRing) & 1) ^ 1, abort_flag)) return false;
  r.slot[s] = x;
  mbar_arrive(&r.full[s]);
  return true;
}

enum Role { kIssue, kOutput, kCompute };
// All threads of the block, whichever role's code they are in.
__device__ inline void block_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// The n-th item for a whole warp; false on a wait that gave up.
__device__ inline bool ring_get(const Ring& r, uint32_t n, int& x, volatile int* abort_flag) {
  const int s = n % kRing;
  if (!warp_wait(&r.full[s], (n / kRing) & 1, abort_flag)) return false;
  x = (int)__reduce_max_sync(0xffffffffu, (unsigned)r.slot[s]);   // the same in every lane, and uniform to the compiler
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[s]);
  return true;
}

// A work item as it is handed out, and where it lies: block `blk` of a sequence of S
// positions whose first is row `row0` of the tensors and place `at` among a head's
// padded rows; head h (of the keys in the dK / dV pass, of the queries in the dQ
// pass).
struct Where {
  int b, h, blk, S, row0;
  long long at;
  int part;                        // dK / dV pass: of the block's query tiles
};
template <bool PACKED>
struct Hand;
template <>
struct Hand<false> {
  using Work = int;
  using Ring = ab::Ring;
  static __device__ inline int draw(const AttnBwdParams&, const Geo&, int, int n) { return n; }
  static __device__ inline bool more(const Geo& g, int x) { return x < g.items; }
  static __device__ inline Where where(const AttnBwdParams& p, const Geo& g, int x, int pass) {
    Where w;
    item_at(p, g, x, pass == 1, w.b, w.h, w.blk);
    w.S = p.S;
    w.row0 = 0;
    w.at = ((long long)w.b * p.H + w.h) * g.sp;
    w.part = 0;
    return w;
  }
};
template <>
struct Hand<true> {
  using Work = packed::Item;
  using Ring = packed::Ring;
  static __device__ inline Work draw(const AttnBwdParams& p, const Geo& g, int pass, int n) {
    return packed::item_at(g.blocks, *g.count, g.order[pass], p.S, BM, n);
  }
  static __device__ inline bool more(const Geo&, const Work& x) { return x.head >= 0; }
  static __device__ inline Where where(const AttnBwdParams&, const Geo& g, const Work& x, int pass) {
    Where w;
    w.b = 0;
    w.h = x.head;
    w.S = x.b.len;
    w.row0 = x.b.start;
    // the last keys of a sequence have the fewest queries: heaviest first from the other end
    w.blk = pass == 0 ? (x.b.len + BM - 1) / BM - 1 - x.b.index : x.b.index;
    w.at = (pass == 0 ? 0 : x.head * g.sp) + x.b.pad;
    w.part = 0;
    if (pass == 0) {
      w.h = x.head / g.parts;
      w.part = x.head - w.h * g.parts;
    }
    return w;
  }
};
// Rows first .. first + R - 1 of the item's sequence, chunk c of head h.
template <bool PACKED, int R>
__device__ inline void load_tile(void* dst, const CUtensorMap* map, uint64_t* bar, int c, int h, const Where& w, int first) {
  if (PACKED) packed::load_rows<R>(dst, map, bar, c, h, packed::Block{w.row0, w.S, 0, 0}, first);
  else tma_load_4d(dst, map, bar, 64 * c, h, first, w.b);
}

// 16 lanes x 16 columns: thread t receives, for n = 0, 1, rows t / 4 (r[4n],
// r[4n + 1]) and t / 4 + 8 (r[4n + 2], r[4n + 3]) of columns 8n + 2 (t % 4) and
// the next.  Issue only, like tmem_ld_32x32b_x16_async.
__device__ inline void tmem_ld_16x256b_x2_async(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ inline void reg_fence8(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
// 16 lanes x 8 columns: thread t gives, for n = 0, 1, rows t / 4 (r[2n]) and
// t / 4 + 8 (r[2n + 1]) of column 4n + t % 4.
__device__ inline void tmem_st_16x128b_x2(uint32_t taddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}
// p <- 2^(s c2 + n) and p <- p (d + n) for two values given as raw fp32 bits
__device__ inline void probs2(float& p0, float& p1, uint32_t s0, uint32_t s1, unsigned long long c2, unsigned long long n) {
  untwo(fma2(two(__uint_as_float(s0), __uint_as_float(s1)), c2, n), p0, p1);
  p0 = ex2_approx(p0);
  p1 = ex2_approx(p1);
}
__device__ inline void dscores2(float& p0, float& p1, uint32_t d0, uint32_t d1, unsigned long long n) {
  untwo(mul2(two(p0, p1), add2(two(__uint_as_float(d0), __uint_as_float(d1)), n)), p0, p1);
}

// 128 rows x 32 bytes of a K-major operand in shared memory to 8 columns of
// tensor memory (a row per lane), in order before later products of this thread.
__device__ inline void tc_cp_128x256b(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}


// The same in fp32, to this lane's row of the shared key's partial sums; `n`, a
// multiple of 8, of its columns exist.
__device__ inline bool store_part(uint32_t taddr, float* dst, float scale, bool row, int n) {
  uint32_t r[2][16], w[32];
  load_32(taddr, r);
  const unsigned long long s2 = two(scale, scale);
  unsigned long long z = 0;
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const unsigned long long v = mul2(two(__uint_as_float(r[x / 8][2 * (x % 8)]), __uint_as_float(r[x / 8][2 * (x % 8) + 1])), s2);
    z = fma2(v, 0, z);
    float v0, v1;
    untwo(v, v0, v1);
    w[2 * x] = __float_as_uint(v0);
    w[2 * x + 1] = __float_as_uint(v1);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (row && 8 * u < n) store_32b(dst + 8 * u, w + 8 * u);
  __syncwarp();
  float z0, z1;
  untwo(z, z0, z1);
  return row && (z0 != 0.f || z1 != 0.f);
}
// ------------------------------------------------------------------- rows
// -delta_i = -sum_c do_ic o_ic (fp32) and nlse_i = -lse_i log2(e) per (b, h, i),
// in rows of `sp` values; rows past the sequence get nlse = -inf (p = 0) and
// delta = 0.  A block takes 16 positions of 8 heads: 16 lanes per row with 8
// features each, the results written through shared memory so that a warp stores
// 16 positions of a head.  Bound by memory: 26.7 us for dense_block's 134 MB (5.0
// TB/s).
constexpr int kRowPos = 16, kRowHeads = 8;
template <bool PACKED>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ AttnBwdParams p, const int sp, const int ni,
                                                   const int nh, const packed::Block* blocks, const int* count) {
  __shared__ float sums[kRowHeads][kRowPos + 1];
  await_previous();
  release_next();
  if (!PACKED && blockIdx.x == 0 && threadIdx.x < 2) p.counter[threadIdx.x] = 0;   // of the launches behind this one
  // block: position group fastest, then head group, then batch; packed: position group
  // of a listed block of 128 rows, then head group
  const int bi = blockIdx.x / ni;
  int i0 = (blockIdx.x - bi * ni) * kRowPos, S = p.S, row0 = 0, pad = 0;
  const int b = PACKED ? 0 : bi / nh, h0 = (bi - b * nh) * kRowHeads;
  if (PACKED) {
    const int e = i0 / BM;
    if (e >= *count) return;
    const int4 at = *reinterpret_cast<const int4*>(blocks + e);
    i0 += (at.z - e) * BM;
    S = at.y;
    row0 = at.x;
    pad = at.w;
  }
  const int sub = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int c0 = sub * 8;
  // row x: head h0 + x % 8 of position i0 + x / 8 (neighbouring heads are
  // neighbours in memory); four rows of a group in flight
#pragma unroll 1
  for (int x0 = group; x0 < kRowPos * kRowHeads; x0 += 64) {
    uint4 a[4], e[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int x = x0 + 16 * n, h = h0 + x % kRowHeads, i = i0 + x / kRowHeads;
      a[n] = e[n] = make_uint4(0, 0, 0, 0);
      if (h < p.H && i < S && c0 < p.d_v) {
        const __nv_bfloat16* o = static_cast<const __nv_bfloat16*>(p.o) + b * p.os[0] + (row0 + i) * p.os[1] + h * p.os[2];
        const __nv_bfloat16* d = static_cast<const __nv_bfloat16*>(p.d_o) + b * p.dos[0] + (row0 + i) * p.dos[1] + h * p.dos[2];
        if (c0 + 8 <= p.d_v) {
          a[n] = *reinterpret_cast<const uint4*>(o + c0);
          e[n] = *reinterpret_cast<const uint4*>(d + c0);
        } else {
          uint32_t wa[4] = {}, we[4] = {};
#pragma unroll
          for (int c = 0; c < 7; ++c)
            if (c0 + c < p.d_v) {
              wa[c / 2] |= (uint32_t)__bfloat16_as_ushort(o[c0 + c]) << (16 * (c % 2));
              we[c / 2] |= (uint32_t)__bfloat16_as_ushort(d[c0 + c]) << (16 * (c % 2));
            }
          a[n] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
          e[n] = make_uint4(we[0], we[1], we[2], we[3]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const uint32_t wa[4] = {a[n].x, a[n].y, a[n].z, a[n].w}, we[4] = {e[n].x, e[n].y, e[n].z, e[n].w};
      float s = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s = fmaf(__uint_as_float(wa[x] << 16), __uint_as_float(we[x] << 16), s);
        s = fmaf(__uint_as_float(wa[x] & 0xffff0000u), __uint_as_float(we[x] & 0xffff0000u), s);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const int x = x0 + 16 * n;
      if (sub == 0) sums[x % kRowHeads][x / kRowHeads] = s;
    }
  }
  __syncthreads();
  const int h = h0 + threadIdx.x / kRowPos, i = i0 + threadIdx.x % kRowPos;
  if (threadIdx.x < kRowPos * kRowHeads && h < p.H && (PACKED || i < sp)) {
    const long long bh = (long long)b * p.H + h, to = bh * sp + pad + i;
    p.ndelta[to] = -sums[threadIdx.x / kRowPos][threadIdx.x % kRowPos];
    p.nlse[to] = i < S ? -p.lse[bh * p.S + row0 + i] * kLog2e : -INFINITY;
  }
}

// ------------------------------------------------------------------ dK, dV
// dS^T (bf16) is written over dP^T, into the first half of each half of its
// columns, so no warp overwrites columns that the other warp of its lanes still
// has to read; P^T lies over S^T in the same way where it has no columns of its
// own.
//
// Per query tile t the tensor core gets dV(t), S(t+1), dK(t), dP(t+1) (S(t+1)
// before dV(t) where P^T is apart: then S(t) need only have been read).  It runs
// the first two while the compute warps turn dP(t) into dS(t), the others while
// they turn S(t+1) into P(t+1).  S(t+1) overwrites P(t) behind dV(t)'s reads of it,
// and dP(t+1) dS(t) behind dK(t)'s, without a wait: the tensor core executes the
// products that one thread issues in their order.  That is how this hardware is
// seen to behave (equal bits on every run, gradients within bounds that a read of
// an overwritten P would break), not what PTX promises: its ordered pairs of
// tcgen05.mma have one accumulator and one shape.  The dQ pass does not rest on it.
//
// The compute warps read S^T and dP^T in the 16 x 256-bit shape (a thread: 4 keys
// x a quarter of the queries): a row value per query then takes 8 bytes per two
// queries and thread from shared memory; with a key's whole row per thread every
// one of these loads was a 16-byte broadcast, 512 bytes of return bandwidth for
// each four queries of each warp, next to the operand reads of the tensor core.
template <int NCH, int NCV, bool PACKED, int ROLE>
__device__ __forceinline__ void dkv_pass(const AttnBwdParams& p, const Maps& mp, const Geo& g, uint8_t* smem, uint64_t* bars,
                                         uint32_t tmem_base, volatile int& abort_flag, int warp, int lane) {
  constexpr int NQ = query_tile(NCH, NCV);
  constexpr bool APART = p_apart(NCH, NCV);
  constexpr int kStages = query_stages(NCH, NCV);
  constexpr int NH = NQ / 2;             // queries per compute warp
  constexpr int NU = NH / 16;            // in units of 16
  constexpr int CQ = NQ * 128;           // bytes of one chunk of a query tile
  uint8_t* kbuf = smem;                                    // NCH chunks
  uint8_t* vbuf = kbuf + NCH * CH;                         // NCV chunks
  uint8_t* qbuf = vbuf + NCV * CH;                         // stages x NCH chunks of a query tile
  uint8_t* dobuf = qbuf + kStages * NCH * CQ;              // stages x NCV chunks
  float* rowv = reinterpret_cast<float*>(dobuf + kStages * NCV * CQ);   // [stage][nlse, -delta][NQ]
  uint64_t* kv_full = bars + 0;
  uint64_t* kv_empty = bars + 1;
  uint64_t* q_full = bars + 2;      // [stages <= 3] Q tile with its nlse and delta
  uint64_t* q_empty = bars + 5;     // [3]
  uint64_t* do_full = bars + 8;     // [3]
  uint64_t* do_empty = bars + 11;   // [3]
  uint64_t* s_full = bars + 14;
  uint64_t* s_empty = bars + 15;
  uint64_t* p_full = bars + 16;
  uint64_t* p_empty = bars + 17;
  uint64_t* dp_full = bars + 18;
  uint64_t* ds_full = bars + 19;
  uint64_t* dv_full = bars + 20;
  uint64_t* dv_empty = bars + 21;
  uint64_t* dk_full = bars + 22;
  uint64_t* dk_empty = bars + 23;
  uint64_t* drain = bars + 24;
  using H = Hand<PACKED>;
  const typename H::Ring ring = {reinterpret_cast<volatile int*>(bars + 34), bars + 25, bars + 29};
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1); mbar_init(kv_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1);
      mbar_init(&do_full[s], 1); mbar_init(&do_empty[s], 1);
    }
    mbar_init(s_full, 1); mbar_init(s_empty, 8);
    mbar_init(p_full, 8); mbar_init(p_empty, 1);
    mbar_init(dp_full, 1); mbar_init(ds_full, 8);
    mbar_init(dv_full, 1); mbar_init(dv_empty, 4);
    mbar_init(dk_full, 1); mbar_init(dk_empty, 4);
    mbar_init(drain, 1);
    for (int s = 0; s < kRing; ++s) { mbar_init(&ring.full[s], 1); mbar_init(&ring.empty[s], 13); }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&mp.q); prefetch_tmap(&mp.k); prefetch_tmap(&mp.v); prefetch_tmap(&mp.d_o);
    if (NCH > g.nck) prefetch_tmap(&mp.ks);
  }
  block_sync();
  const uint32_t t_dk = tmem_base, t_dv = t_dk + 64 * NCH, t_s = t_dv + 64 * NCV, t_dp = t_s + NQ, t_p = APART ? t_dp + NQ : t_s;
  constexpr uint32_t kHalfP = APART ? NH / 2 : NH;       // second half of the queries in P^T
  auto fail = [&]() { abort_flag = 1; set_status(p.status, MC_STATUS_TIMEOUT); };
  // first query tile that has a query at or behind the block's first key, and the
  // number of the sequence's tiles
  auto first_tile = [&](int blk) { return p.causal ? (blk * BM) / NQ : 0; };
  auto end_tile = [&](const Where& w) { return PACKED ? (w.S + NQ - 1) / NQ : g.nt; };
  // The item's query tiles: n of those from t0 to end of every head of the group, from
  // the lo-th on.
  struct Span {
    int t0, end, lo, n, parts;
  };
  auto span_of = [&](const Where& w) {
    Span a;
    a.t0 = first_tile(w.blk);
    a.end = end_tile(w);
    a.lo = 0;
    a.n = a.end - a.t0;
    a.parts = 1;
    if (PACKED) {
      a.n *= g.q_heads;
      if (g.parts > 1) {
        const int all = a.n, per = max((all + g.parts - 1) / g.parts, kPartTiles);
        a.parts = (all + per - 1) / per;
        a.lo = w.part * per;
        a.n = min(per, all - a.lo);          // none: no such part
      }
    }
    return a;
  };

  if (ROLE == kIssue && warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t li = 0, s = 0, ph = 0;
      bool used_kv = false, used_q[kStages] = {}, used_do[kStages] = {};
      uint32_t par_kv = 0, par_q[kStages] = {}, par_do[kStages] = {};
      int next = atomicAdd(p.counter, 1);
      auto draw = [&]() {                      // the counter's item, or the next one that has tiles
        typename H::Work d = H::draw(p, g, 0, next);
        if (PACKED)
          while (H::more(g, d) && span_of(H::where(p, g, d, 0)).n <= 0) {
            next = atomicAdd(p.counter, 1);
            d = H::draw(p, g, 0, next);
          }
        return d;
      };
      typename H::Work x = draw(), x1 = x;
      bool ok = ring_put(ring, 0, x, &abort_flag);
      for (uint32_t n = 1; ok && H::more(g, x); x = x1, ++n) {
        const Where w = H::where(p, g, x, 0);
        const Span a = span_of(w);
        const int t0 = a.t0, end = a.end;
        int left = a.n;                        // tiles of the item
        int hh = PACKED ? a.lo / (end - t0) : 0;
        bool first = true;
        for (int it = t0 + a.lo - hh * (end - t0); left > 0; --left, first = false, it = it + 1 < end ? it + 1 : (++hh, t0)) {
          const int h = PACKED ? w.h * g.q_heads + hh : w.h;
          const long long rowbase = PACKED ? h * g.sp + w.at : w.at;
          if (left == 2 || (left == 1 && first)) next = atomicAdd(p.counter, 1);       // used a tile later: its latency is hidden
          if (left == 1) {
            x1 = draw();
            if (!ring_put(ring, n, x1, &abort_flag)) { ok = false; break; }
          }
          if (!mbar_wait(&q_empty[s], ph ^ 1, &abort_flag)) { ok = false; break; }
          mbar_arrive_expect_tx(&q_full[s], NCH * CQ + 2 * NQ * 4);
          for (int c = 0; c < NCH; ++c) load_tile<PACKED, NQ>(qbuf + (s * NCH + c) * CQ, &mp.q, &q_full[s], c, h, w, it * NQ);
          bulk_load_1d(rowv + s * 2 * NQ, p.nlse + rowbase + it * NQ, NQ * 4, &q_full[s]);
          bulk_load_1d(rowv + s * 2 * NQ + NQ, p.ndelta + rowbase + it * NQ, NQ * 4, &q_full[s]);
          used_q[s] = true; par_q[s] = ph;
          if (!mbar_wait(&do_empty[s], ph ^ 1, &abort_flag)) { ok = false; break; }
          mbar_arrive_expect_tx(&do_full[s], NCV * CQ);
          for (int c = 0; c < NCV; ++c) load_tile<PACKED, NQ>(dobuf + (s * NCV + c) * CQ, &mp.d_o, &do_full[s], c, h, w, it * NQ);
          used_do[s] = true; par_do[s] = ph;
          if (++s == kStages) { s = 0; ph ^= 1; }
          if (first) {           // the item's keys and values, behind its first query tile
            if (!mbar_wait(kv_empty, (li & 1) ^ 1, &abort_flag)) { ok = false; break; }
            mbar_arrive_expect_tx(kv_full, (NCH + NCV) * CH);
            for (int c = 0; c < NCH; ++c) {
              if (PACKED || c < g.nck) load_tile<PACKED, BM>(kbuf + c * CH, &mp.k, kv_full, c, w.h, w, w.blk * BM);
              else tma_load_3d(kbuf + c * CH, &mp.ks, kv_full, 64 * (c - g.nck), w.blk * BM, w.b);
            }
            for (int c = 0; c < NCV; ++c) load_tile<PACKED, BM>(vbuf + c * CH, &mp.v, kv_full, c, w.h, w, w.blk * BM);
            used_kv = true; par_kv = li & 1;
          }
        }
        ++li;
      }
      if (!ok) fail();
      // every issued copy must have landed before the CTA may exit
      if (used_kv) mbar_wait(kv_full, par_kv, nullptr);
      for (int i = 0; i < kStages; ++i) {
        if (used_q[i]) mbar_wait(&q_full[i], par_q[i], nullptr);
        if (used_do[i]) mbar_wait(&do_full[i], par_do[i], nullptr);
      }
    }
  } else if (ROLE == kIssue && warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = make_idesc_bf16(BM, NQ, 0, 0);
    constexpr uint32_t idesc_dv = make_idesc_bf16(BM, 64 * NCV, 0, 1);
    constexpr uint32_t idesc_dk = make_idesc_bf16(BM, 64 * NCH, 0, 1);
    // operand descriptors: rows of 64 features, K-major for S^T and dP^T,
    // MN-major (16 query rows = 2048 bytes per k-step) for dV and dK
    const uint64_t dk_ = make_sdesc_sw128(smem_u32(kbuf), 16, 1024), dv_ = make_sdesc_sw128(smem_u32(vbuf), 16, 1024);
    const uint64_t dq_ = make_sdesc_sw128(smem_u32(qbuf), 16, 1024), ddo_ = make_sdesc_sw128(smem_u32(dobuf), 16, 1024);
    const uint64_t mq_ = make_sdesc(smem_u32(qbuf), CQ, 1024, 2), mdo_ = make_sdesc(smem_u32(dobuf), CQ, 1024, 2);
    uint32_t t = 0, li = 0;
    // stages: of the next S, the next dP, and the tile whose dV and dK come next
    uint32_t ss = 0, sph = 0, sp = 0, pph = 0, sd = 0;
    bool issued = false;
    auto scores = [&]() -> bool {          // S^T = K Q^T
      if (!warp_wait(&q_full[ss], sph, &abort_flag)) return false;
      tc_fence_after();
      const uint64_t q0 = dq_ + ss * (NCH * CQ / 16);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4 * NCH; ++c)
          tc_mma(t_s, dk_ + ((c >> 2) * CH + (c & 3) * 32) / 16, q0 + ((c >> 2) * CQ + (c & 3) * 32) / 16, idesc_s, c > 0);
        tc_commit(s_full);
      }
      __syncwarp();
      if (++ss == kStages) { ss = 0; sph ^= 1; }
      return true;
    };
    auto dprobs = [&](bool last) -> bool { // dP^T = V dO^T; `last`: keys and values are free after it
      if (!warp_wait(&do_full[sp], pph, &abort_flag)) return false;
      tc_fence_after();
      const uint64_t d0 = ddo_ + sp * (NCV * CQ / 16);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4 * NCV; ++c)
          tc_mma(t_dp, dv_ + ((c >> 2) * CH + (c & 3) * 32) / 16, d0 + ((c >> 2) * CQ + (c & 3) * 32) / 16, idesc_s, c > 0);
        tc_commit(dp_full);
        if (last) tc_commit(kv_empty);
      }
      __syncwarp();
      if (++sp == kStages) { sp = 0; pph ^= 1; }
      return true;
    };
    // A (tensor memory): NQ / 16 k-steps of 8 columns; the second half of the
    // queries starts at column a + `half`
    auto accumulate = [&](uint32_t d, uint32_t a, int half, uint64_t b0, uint32_t idesc, bool add, uint64_t* done,
                          uint64_t* done2, uint64_t* done3) {
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < NQ / 16; ++kk)
          tc_mma_ts(d, a + (kk < NU ? kk * 8 : half + (kk - NU) * 8), b0 + kk * 128, idesc, (add || kk > 0) ? 1u : 0u);
        tc_commit(done);
        if (done2) tc_commit(done2);
        if (done3) tc_commit(done3);
      }
      __syncwarp();
    };
    for (;; ) {
      typename H::Work x;
      if (!ring_get(ring, li, x, &abort_flag)) { fail(); break; }
      if (!H::more(g, x)) break;
      const Where w = H::where(p, g, x, 0);
      const int nt = span_of(w).n;
      // S and dP of the previous item have been read: its last p_full and
      // ds_full were waited for below
      bool ok = warp_wait(kv_full, li & 1, &abort_flag) && scores();
      if (!ok) { fail(); break; }
      issued = true;
      if (!dprobs(nt == 1)) { fail(); break; }
      for (int i = 0; i < nt; ++i, ++t) {
        if (APART && !warp_wait(s_empty, t & 1, &abort_flag)) { ok = false; break; }
        if (APART && i + 1 < nt && !scores()) { ok = false; break; }
        if (!warp_wait(p_full, t & 1, &abort_flag)) { ok = false; break; }
        if (i == 0 && !warp_wait(dv_empty, (li & 1) ^ 1, &abort_flag)) { ok = false; break; }
        tc_fence_after();
        accumulate(t_dv, t_p, kHalfP, mdo_ + sd * (NCV * CQ / 16), idesc_dv, i > 0, &do_empty[sd],
                   APART ? p_empty : nullptr, i + 1 == nt ? dv_full : nullptr);
        if (!APART && i + 1 < nt && !scores()) { ok = false; break; }
        if (!warp_wait(ds_full, t & 1, &abort_flag)) { ok = false; break; }
        if (i == 0 && !warp_wait(dk_empty, (li & 1) ^ 1, &abort_flag)) { ok = false; break; }
        tc_fence_after();
        accumulate(t_dk, t_dp, NH, mq_ + sd * (NCH * CQ / 16), idesc_dk, i > 0, &q_empty[sd], nullptr,
                   i + 1 == nt ? dk_full : nullptr);
        if (++sd == kStages) sd = 0;
        if (i + 1 < nt && !dprobs(i + 2 == nt)) { ok = false; break; }
      }
      if (!ok) { fail(); break; }
      ++li;
    }
    if (issued) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, nullptr);
    }
  } else if (PACKED && ROLE == kIssue) {
    // ------------------------------------------------------------ rows of no sequence
    const packed::Outside out = packed::outside_of(g.count, p.S);
    const int w = 2 * blockIdx.x + warp - 2, warps = 2 * gridDim.x, kv = p.H / g.q_heads;
    if (g.fill & MC_FILL_DQ) packed::fill_rows(out, p.dq, p.dqs + 1, p.H, p.d_head, w, warps);
    if (g.fill & MC_FILL_DK) packed::fill_rows(out, p.dk, p.dks + 1, kv, p.d_head, w, warps);
    if (g.fill & MC_FILL_DV) packed::fill_rows(out, p.dv, p.dvs + 1, kv, p.d_v, w, warps);
  } else if (ROLE == kOutput) {
    // ------------------------------------------------------------ output
    // Warp w: keys 32 q .. 32 q + 31 of the block, every column: dV as soon as the
    // item's last dV product is done, then scale * dK (the shared key's columns go
    // to the per-head fp32 partial sums), while the other warps are at the next
    // item.
    const int q = warp & 3;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const bool wide_v = rows_wide(p.dv, p.dvs), wide_k = rows_wide(p.dk, p.dks);
    uint32_t li = 0;
    bool bad = false, ok = true;
    for (;; ++li) {
      typename H::Work x;
      if (!(ok = ring_get(ring, li, x, &abort_flag)) || !H::more(g, x)) break;
      const Where w = H::where(p, g, x, 0);
      const int b = w.b, h = w.h, key = w.blk * BM + q * 32 + lane;
      const bool row = key < w.S;
      __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.dv) + b * p.dvs[0] + (w.row0 + key) * p.dvs[1] + h * p.dvs[2];
      __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(p.dk) + b * p.dks[0] + (w.row0 + key) * p.dks[1] + h * p.dks[2];
      // one of several parts: fp32 rows of dV, then dK, that join_kernel adds up
      const bool parted = PACKED && g.parts > 1 && span_of(w).parts > 1;
      float* part = PACKED ? p.part + (((long long)h * g.parts + w.part) * p.S + w.row0 + key) * packed_part_pitch(p.d_head, p.d_v) : nullptr;
#pragma unroll 1
      for (int c = 0; c < 2 * (NCV + NCH); ++c) {
        const bool is_v = c < 2 * NCV;
        if (c == 0 || c == 2 * NCV) {
          ok = warp_wait(is_v ? dv_full : dk_full, li & 1, &abort_flag);
          if (!ok) break;
          tc_fence_after();
        }
        const int col = 32 * (is_v ? c : c - 2 * NCV);
        const uint32_t from = (is_v ? t_dv : t_dk) + lanes + col;
        if (is_v || PACKED || col < 64 * g.nck) {
          const int n = (is_v ? p.d_v : p.d_head) - col;
          if (n > 0) {
            if (parted) bad |= store_part(from, part + (is_v ? 0 : part_pitch(p.d_v)) + col, is_v ? 1.f : p.scale, row, n);
            else bad |= store_rows(from, (is_v ? dv : dk) + col, is_v ? 1.f : p.scale, row, is_v ? wide_v : wide_k, n);
          }
        } else {
          const int f0 = col - p.d_head, n = part_pitch(p.d_shared) - f0;
          if (n > 0)
            bad |= store_part(from, p.part + (((long long)b * p.H + h) * p.S + key) * part_pitch(p.d_shared) + f0, p.scale, row, n);
        }
        if (c == 2 * NCV - 1 || c == 2 * (NCV + NCH) - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(is_v ? dv_empty : dk_empty);
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) fail();
    if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, MC_STATUS_NONFINITE_UPDATE);
  } else if (ROLE == kCompute) {
    // ------------------------------------------------------------ P, dS
    // Warp e = warp - 8: keys 32 q .. 32 q + 31 of the block (q = warp & 3, its
    // TMEM lane quadrant), queries of half e >> 2 of the tile.  A thread holds
    // keys r0, r0 + 8, r0 + 16, r0 + 24 and, of each 8 queries, the two from c0.
    const int q = warp & 3, hf = (warp - 8) >> 2;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t ts = t_s + lanes + hf * NH, tdp = t_dp + lanes + hf * NH, tp = t_p + lanes + hf * kHalfP;
    const int r0 = lane >> 2, c0 = 2 * (lane & 3);
    const float c2 = p.scale * kLog2e;
    const unsigned long long c22 = two(c2, c2);
    uint32_t t = 0, li = 0, s = 0, sph = 0;
    for (;; ) {
      typename H::Work x;
      if (!ring_get(ring, li, x, &abort_flag)) { fail(); break; }
      if (!H::more(g, x)) break;
      const Where w = H::where(p, g, x, 0);
      const Span a = span_of(w);
      const int t0 = a.t0, end = a.end;
      bool ok = true;
      int left = a.n;
      for (int it = PACKED ? t0 + a.lo % (end - t0) : t0; left > 0; --left, it = it + 1 < end ? it + 1 : t0, ++t) {
        const float* nl = rowv + s * 2 * NQ + hf * NH + c0;
        const int i0 = it * NQ + hf * NH;
        const int key0 = w.blk * BM + q * 32;
        const bool diag = p.causal && i0 < key0 + 31;    // some (i, j) of the warp has i < j
        ok = warp_wait(&q_full[s], sph, &abort_flag) && warp_wait(s_full, t & 1, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        float pv[NU][2][8];              // [unit][16-key half][register of the 16 x 256-bit shape]
        {
          uint32_t r[NU][2][8];
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) tmem_ld_16x256b_x2_async(ts + ((uint32_t)(16 * hh) << 16) + u * 16, r[u][hh]);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) reg_fence8(r[u][hh]);
          if (APART) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_empty);
          }
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const unsigned long long l = *reinterpret_cast<const unsigned long long*>(nl + u * 16 + m * 8);
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int x = 4 * m; x < 4 * m + 4; x += 2)
                  probs2(pv[u][hh][x], pv[u][hh][x + 1], r[u][hh][x], r[u][hh][x + 1], c22, l);
            }
        }
        if (diag) {
          // register x of unit u, half hh: query i0 + 16 u + 8 (x / 4) + c0 + x % 2,
          // key key0 + 16 hh + 8 (x / 2 % 2) + r0
          const int d = i0 + c0 - key0 - r0;
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (d + 16 * u + 8 * (x / 4) + x % 2 - 16 * hh - 8 * (x / 2 % 2) < 0) pv[u][hh][x] = 0.f;
        }
        if (APART) {
          ok = warp_wait(p_empty, (t & 1) ^ 1, &abort_flag);     // dV(t-1) has read P(t-1)
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float* v = pv[u][hh];
            tmem_st_16x128b_x2(tp + ((uint32_t)(16 * hh) << 16) + u * 8, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
          }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        // a query that sees one key: its softmax is 1 whatever the logit, and ds is 0 (the
        // dense sequences short enough to notice take a kernel of their own)
        if (PACKED && i0 + c0 == 0) pv[0][0][0] = pv[0][0][2] = pv[0][1][0] = pv[0][1][2] = 0.f;

        ok = warp_wait(dp_full, t & 1, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        // unit by unit, the next one's load under the arithmetic: dS^T of unit u
        // (8 columns) lies before every column that is still to be read
        uint32_t r[2][2][8];
        auto load = [&](int u) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) tmem_ld_16x256b_x2_async(tdp + ((uint32_t)(16 * hh) << 16) + u * 16, r[u & 1][hh]);
        };
        load(0);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          tmem_ld_wait();
          reg_fence8(r[u & 1][0]);
          reg_fence8(r[u & 1][1]);
          if (u + 1 < NU) load(u + 1);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const unsigned long long d = *reinterpret_cast<const unsigned long long*>(nl + NQ + u * 16 + m * 8);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int x = 4 * m; x < 4 * m + 4; x += 2)
                dscores2(pv[u][hh][x], pv[u][hh][x + 1], r[u & 1][hh][x], r[u & 1][hh][x + 1], d);
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float* v = pv[u][hh];
            tmem_st_16x128b_x2(tdp + ((uint32_t)(16 * hh) << 16) + u * 8, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
        if (++s == kStages) { s = 0; sph ^= 1; }
      }
      if (!ok) { if (lane == 0) fail(); break; }
      ++li;
    }
  }

  // everything in flight has landed and been read: the next pass may reuse tensor
  // memory and shared memory (its barriers have memory of their own)
  fence_async_smem();
  tc_fence_before();
  block_sync();
  tc_fence_after();
}

// --------------------------------------------------------------------- dQ
// Q and dO are the A operands of every product of an item but one, so they move
// from shared memory to tensor memory once per item (tcgen05.cp, a 16-feature
// k-step at a time) and only keys and values are read from shared memory for the
// products: with Q and dO there too, a product of 64 keys took 48 clocks instead of
// 32, and the whole call 734 / 1030 us instead of 715 / 997 on dense_block /
// k2_mla_layer (as both passes then were).
//
// dS has columns of its own, so S(t+1) starts as soon as S(t) has been read and
// dP(t+1) as soon as dP(t) has.  Issue order per key tile t: S(t+1) | dP(t+1),
// dQ(t).  A key tile is held from S(t) to dQ(t), two products later than the next
// one's S wants its own, so keys have three stages, and values where they fit.
template <int NCH, int NCV, bool PACKED, int ROLE>
__device__ __forceinline__ void dq_pass(const AttnBwdParams& p, const Maps& mp, const Geo& g, uint8_t* smem, uint64_t* bars,
                                         uint32_t tmem_base, volatile int& abort_flag, int warp, int lane) {
  constexpr int BN = key_tile(NCH, NCV), NH = BN / 2;
  constexpr int kStages = kKeyStages, VS = value_stages(NCH, NCV);
  constexpr int QT = q_in_tmem(NCH);     // chunks of Q that are operands in tensor memory
  constexpr bool DOT = do_in_tmem(NCH);  // dO is one too
  constexpr int CK = BN * 128;           // bytes of one chunk of a key tile
  uint8_t* qbuf = smem;                                 // NCH chunks
  uint8_t* dobuf = qbuf + NCH * CH;                     // NCV chunks
  uint8_t* kbuf = dobuf + NCV * CH;                     // 3 x NCH chunks of a key tile
  uint8_t* vbuf = kbuf + kStages * NCH * CK;            // VS x NCV chunks
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;      // [3]
  uint64_t* k_empty = bars + 5;     // [3]
  uint64_t* v_full = bars + 8;      // [3]
  uint64_t* v_empty = bars + 11;    // [3]
  uint64_t* s_full = bars + 14;
  uint64_t* s_empty = bars + 15;
  uint64_t* dp_full = bars + 16;
  uint64_t* ds_full = bars + 17;
  uint64_t* ds_empty = bars + 18;
  uint64_t* acc_full = bars + 19;
  uint64_t* acc_empty = bars + 20;
  uint64_t* drain = bars + 21;
  uint64_t* do_full = bars + 33;
  uint64_t* do_empty = bars + 34;
  using H = Hand<PACKED>;
  const typename H::Ring ring = {reinterpret_cast<volatile int*>(bars + (PACKED ? 36 : 31)), bars + 22, bars + 26};
  static_assert(36 * 8 + packed::kRing * packed::kSlot * 4 <= kBarBytes, "barriers");
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1); mbar_init(q_empty, 1); mbar_init(do_full, 1); mbar_init(do_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1);     // VS of them are used
    }
    mbar_init(s_full, 1); mbar_init(s_empty, 8);
    mbar_init(dp_full, 1); mbar_init(ds_full, 8); mbar_init(ds_empty, 1);
    mbar_init(acc_full, 1); mbar_init(acc_empty, 4);
    mbar_init(drain, 1);
    for (int s = 0; s < kRing; ++s) { mbar_init(&ring.full[s], 1); mbar_init(&ring.empty[s], 13); }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&mp.q); prefetch_tmap(&mp.k); prefetch_tmap(&mp.v); prefetch_tmap(&mp.d_o);
    if (NCH > g.nck) prefetch_tmap(&mp.ks);
  }
  block_sync();
  const uint32_t t_dq = tmem_base, t_q = t_dq + 64 * NCH, t_do = t_q + 32 * QT, t_s = t_do + (DOT ? 32 * NCV : 0), t_dp = t_s + BN,
                 t_ds = t_dp + BN;
  auto fail = [&]() { abort_flag = 1; set_status(p.status, MC_STATUS_TIMEOUT); };
  auto tiles = [&](const Where& w) {
    const int hi = p.causal ? min(w.S, (w.blk + 1) * BM) : w.S;
    return (hi + BN - 1) / BN;
  };

  if (ROLE == kIssue && warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t li = 0, s = 0, ph = 0, sv = 0, phv = 0;
      bool used_q = false, used_do = false, used_k[kStages] = {}, used_v[VS] = {};
      uint32_t par_q = 0, par_do = 0, par_k[kStages] = {}, par_v[VS] = {};
      int next = atomicAdd(p.counter + 1, 1);
      typename H::Work x = H::draw(p, g, 1, next), x1 = x;
      bool ok = ring_put(ring, 0, x, &abort_flag);
      for (uint32_t n = 1; ok && H::more(g, x); x = x1, ++n) {
        const Where w = H::where(p, g, x, 1);
        const int nt = tiles(w), kh = PACKED ? w.h / g.q_heads : w.h;      // the head of its keys
        // the queries' buffer is free once the item before has begun
        if (!mbar_wait(q_empty, (li & 1) ^ 1, &abort_flag)) { ok = false; break; }
        mbar_arrive_expect_tx(q_full, NCH * CH);
        for (int c = 0; c < NCH; ++c) load_tile<PACKED, BM>(qbuf + c * CH, &mp.q, q_full, c, w.h, w, w.blk * BM);
        used_q = true; par_q = li & 1;
        auto load_do = [&]() -> bool {
          if (!mbar_wait(do_empty, (li & 1) ^ 1, &abort_flag)) return false;
          mbar_arrive_expect_tx(do_full, NCV * CH);
          for (int c = 0; c < NCV; ++c) load_tile<PACKED, BM>(dobuf + c * CH, &mp.d_o, do_full, c, w.h, w, w.blk * BM);
          used_do = true; par_do = li & 1;
          return true;
        };
        if (DOT && !load_do()) { ok = false; break; }
        for (int it = 0; it < nt; ++it) {
          if (it == max(0, nt - 2)) next = atomicAdd(p.counter + 1, 1);    // used a tile later: its latency is hidden
          if (it == nt - 1) {
            x1 = H::draw(p, g, 1, next);
            if (!ring_put(ring, n, x1, &abort_flag)) { ok = false; break; }
          }
          if (!mbar_wait(&k_empty[s], ph ^ 1, &abort_flag)) { ok = false; break; }
          mbar_arrive_expect_tx(&k_full[s], NCH * CK);
          for (int c = 0; c < NCH; ++c) {
            uint8_t* dst = kbuf + (s * NCH + c) * CK;
            if (PACKED || c < g.nck) load_tile<PACKED, BN>(dst, &mp.k, &k_full[s], c, kh, w, it * BN);
            else tma_load_3d(dst, &mp.ks, &k_full[s], 64 * (c - g.nck), it * BN, w.b);
          }
          used_k[s] = true; par_k[s] = ph;
          if (++s == kStages) { s = 0; ph ^= 1; }
          if (!DOT && it == 0 && !load_do()) { ok = false; break; }        // not needed before the first S
          if (!mbar_wait(&v_empty[sv], phv ^ 1, &abort_flag)) { ok = false; break; }
          mbar_arrive_expect_tx(&v_full[sv], NCV * CK);
          for (int c = 0; c < NCV; ++c) load_tile<PACKED, BN>(vbuf + (sv * NCV + c) * CK, &mp.v, &v_full[sv], c, kh, w, it * BN);
          used_v[sv] = true; par_v[sv] = phv;
          if (++sv == VS) { sv = 0; phv ^= 1; }
        }
        ++li;
      }
      if (!ok) fail();
      if (used_q) mbar_wait(q_full, par_q, nullptr);
      if (used_do) mbar_wait(do_full, par_do, nullptr);
      for (int i = 0; i < kStages; ++i)
        if (used_k[i]) mbar_wait(&k_full[i], par_k[i], nullptr);
      for (int i = 0; i < VS; ++i)
        if (used_v[i]) mbar_wait(&v_full[i], par_v[i], nullptr);
    }
  } else if (ROLE == kIssue && warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = make_idesc_bf16(BM, BN, 0, 0);
    constexpr uint32_t idesc_dq = make_idesc_bf16(BM, 64 * NCH, 0, 1);
    const uint64_t dq_ = make_sdesc_sw128(smem_u32(qbuf), 16, 1024), ddo_ = make_sdesc_sw128(smem_u32(dobuf), 16, 1024);
    const uint64_t dk_ = make_sdesc_sw128(smem_u32(kbuf), 16, 1024), dv_ = make_sdesc_sw128(smem_u32(vbuf), 16, 1024);
    const uint64_t mk_ = make_sdesc(smem_u32(kbuf), CK, 1024, 2);
    uint32_t t = 0, li = 0, ks = 0, kph = 0, vs = 0, vph = 0, kd = 0;   // tiles, items; stages of S, of dP and of dQ
    bool issued = false;
    auto scores = [&](bool last) -> bool { // S = Q K^T; `last`: Q is free after it
      if (!warp_wait(&k_full[ks], kph, &abort_flag)) return false;
      tc_fence_after();
      const uint64_t k0 = dk_ + ks * (NCH * CK / 16);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4 * NCH; ++c)
          if (c < 4 * QT) tc_mma_ts(t_s, t_q + c * 8, k0 + ((c >> 2) * CK + (c & 3) * 32) / 16, idesc_s, c > 0);
          else tc_mma(t_s, dq_ + ((c >> 2) * CH + (c & 3) * 32) / 16, k0 + ((c >> 2) * CK + (c & 3) * 32) / 16, idesc_s, 1);
        tc_commit(s_full);
        if (QT < NCH && last) tc_commit(q_empty);
      }
      __syncwarp();
      if (++ks == kStages) { ks = 0; kph ^= 1; }
      return true;
    };
    auto dprobs = [&](bool last) -> bool { // dP = dO V^T; `last`: dO is free after it
      if (!warp_wait(&v_full[vs], vph, &abort_flag)) return false;
      tc_fence_after();
      const uint64_t v0 = dv_ + vs * (NCV * CK / 16);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4 * NCV; ++c)
          if (DOT) tc_mma_ts(t_dp, t_do + c * 8, v0 + ((c >> 2) * CK + (c & 3) * 32) / 16, idesc_s, c > 0);
          else tc_mma(t_dp, ddo_ + ((c >> 2) * CH + (c & 3) * 32) / 16, v0 + ((c >> 2) * CK + (c & 3) * 32) / 16, idesc_s, c > 0);
        tc_commit(&v_empty[vs]);
        tc_commit(dp_full);
        if (!DOT && last) tc_commit(do_empty);
      }
      __syncwarp();
      if (++vs == VS) { vs = 0; vph ^= 1; }
      return true;
    };
    for (;; ) {
      typename H::Work x;
      if (!ring_get(ring, li, x, &abort_flag)) { fail(); break; }
      if (!H::more(g, x)) break;
      const int nt = tiles(H::where(p, g, x, 1));
      // The previous item's S and dP are done and have been read: its last
      // s_empty and ds_full were waited for below.  So its queries may be
      // overwritten.
      bool ok = warp_wait(q_full, li & 1, &abort_flag) && (!DOT || warp_wait(do_full, li & 1, &abort_flag));
      if (!ok) { fail(); break; }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4 * QT; ++c) tc_cp_128x256b(t_q + c * 8, dq_ + ((c >> 2) * CH + (c & 3) * 32) / 16);
#pragma unroll
        for (int c = 0; c < 4 * NCV; ++c)
          if (DOT) tc_cp_128x256b(t_do + c * 8, ddo_ + ((c >> 2) * CH + (c & 3) * 32) / 16);
        if (QT == NCH) tc_commit(q_empty);
        if (DOT) tc_commit(do_empty);
      }
      __syncwarp();
      issued = true;
      if (!scores(nt == 1) || !(DOT || warp_wait(do_full, li & 1, &abort_flag)) || !dprobs(nt == 1)) { fail(); break; }
      for (int i = 0; i < nt; ++i, ++t) {
        if (!warp_wait(s_empty, t & 1, &abort_flag)) { ok = false; break; }
        if (i + 1 < nt && !scores(i + 2 == nt)) { ok = false; break; }
        if (!warp_wait(ds_full, t & 1, &abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (i + 1 < nt && !dprobs(i + 2 == nt)) { ok = false; break; }
        if (i == 0 && !warp_wait(acc_empty, (li & 1) ^ 1, &abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint64_t k0 = mk_ + kd * (NCH * CK / 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            tc_mma_ts(t_dq, t_ds + kk * 8, k0 + kk * 128, idesc_dq, (i > 0 || kk > 0) ? 1u : 0u);
          tc_commit(&k_empty[kd]);
          tc_commit(ds_empty);
        }
        __syncwarp();
        if (++kd == kStages) kd = 0;
      }
      if (!ok) { fail(); break; }
      if (elect_one()) tc_commit(acc_full);
      __syncwarp();
      ++li;
    }
    if (issued) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, nullptr);
    }
  } else if (ROLE == kOutput) {
    // ------------------------------------------------------------ output
    // Warp w: queries 32 q .. 32 q + 31 of the block: scale * dQ, while the other
    // warps are at the next item
    const int q = warp & 3, D = p.d_head + p.d_shared;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const bool wide = rows_wide(p.dq, p.dqs);
    bool bad = false, ok = true;
    for (uint32_t li = 0;; ++li) {
      typename H::Work x;
      if (!(ok = ring_get(ring, li, x, &abort_flag)) || !H::more(g, x)) break;
      const Where w = H::where(p, g, x, 1);
      if (!(ok = warp_wait(acc_full, li & 1, &abort_flag))) break;
      tc_fence_after();
      const int i = w.blk * BM + q * 32 + lane;
      __nv_bfloat16* dq = static_cast<__nv_bfloat16*>(p.dq) + w.b * p.dqs[0] + (w.row0 + i) * p.dqs[1] + w.h * p.dqs[2];
#pragma unroll 1
      for (int col = 0; col < D; col += 32)
        bad |= store_rows(t_dq + lanes + col, dq + col, p.scale, i < w.S, wide, D - col);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
    }
    if (!ok && lane == 0) fail();
    if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, MC_STATUS_NONFINITE_UPDATE);
  } else if (ROLE == kCompute) {
    // ------------------------------------------------------------ P, dS
    const int q = warp & 3, hf = (warp - 8) >> 2;
    const int row = q * 32 + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t ts = t_s + lanes + hf * NH, tdp = t_dp + lanes + hf * NH, tds = t_ds + lanes + hf * (NH / 2);
    const float c2 = p.scale * kLog2e;
    const unsigned long long c22 = two(c2, c2);
    uint32_t t = 0, li = 0;
    // this item and the next one, whose row values are loaded an item ahead
    Where w, w1 = {};
    float nl = 0.f, dl = 0.f, nl1 = 0.f, dl1 = 0.f;
    bool more = true;
    auto fetch = [&](uint32_t n) -> bool {   // item n: coordinates, nlse and delta of this thread's query
      typename H::Work x;
      if (!ring_get(ring, n, x, &abort_flag)) return false;
      more = H::more(g, x);
      if (more) {
        w1 = H::where(p, g, x, 1);
        const long long at = w1.at + w1.blk * BM + row;   // inside: places are padded to whole blocks
        nl1 = p.nlse[at];
        dl1 = p.ndelta[at];
      }
      return true;
    };
    bool ok = fetch(0);
    while (ok && more) {
      w = w1; nl = nl1; dl = dl1;
      const unsigned long long nl2 = two(nl, nl), dl2 = two(dl, dl);
      const int blk = w.blk, i = blk * BM + row;         // this thread's query
      const int nt = tiles(w);
      for (int it = 0; it < nt; ++it, ++t) {
        const int j0 = it * BN + hf * NH;
        const bool full = j0 + NH <= w.S && (!p.causal || j0 + NH - 1 <= blk * BM + q * 32);
        if (it == nt - 1 && !(ok = fetch(li + 1))) break;
        ok = warp_wait(s_full, t & 1, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        float pv[NH];
        {
          uint32_t r[NH / 16][16];
#pragma unroll
          for (int c = 0; c < NH / 16; ++c) tmem_ld_32x32b_x16_async(ts + c * 16, r[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < NH / 16; ++c) reg_fence16(r[c]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_empty);
#pragma unroll
          for (int x = 0; x < NH; x += 2) probs2(pv[x], pv[x + 1], r[x / 16][x % 16], r[x / 16][x % 16 + 1], c22, nl2);
        }
        ok = warp_wait(dp_full, t & 1, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        {
          uint32_t r[NH / 16][16];
#pragma unroll
          for (int c = 0; c < NH / 16; ++c) tmem_ld_32x32b_x16_async(tdp + c * 16, r[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < NH / 16; ++c) reg_fence16(r[c]);
#pragma unroll
          for (int x = 0; x < NH; x += 2) dscores2(pv[x], pv[x + 1], r[x / 16][x % 16], r[x / 16][x % 16 + 1], dl2);
        }
        if (!full) {
          // last key of this row; where there is only one, none: as in the dK / dV pass
          const int lim = PACKED && i == 0 ? -1 : p.causal ? min(i, w.S - 1) : w.S - 1;
#pragma unroll
          for (int x = 0; x < NH; ++x)
            if (j0 + x > lim) pv[x] = 0.f;
        }
        ok = warp_wait(ds_empty, (t & 1) ^ 1, &abort_flag);      // dQ(t-1) has read dS(t-1)
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NH / 16; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) pk[x] = pack_bf16(pv[c * 16 + 2 * x], pv[c * 16 + 2 * x + 1]);
          tmem_st_32x32b_x8(tds + c * 8, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      ++li;
    }
    if (!ok && lane == 0) fail();
  }

  // everything in flight has landed and been read: the next pass may reuse tensor
  // memory and shared memory (its barriers have memory of their own)
  fence_async_smem();
  tc_fence_before();
  block_sync();
  tc_fence_after();
}

// ---------------------------------------------------------------- both passes
// One persistent CTA per SM takes dK / dV items until there are none, then dQ
// items: the second pass starts wherever the first one has run out, with no
// launch in between, and a small batch runs both at once on different SMs.  (As
// two launches: 623 us instead of 614 on dense_block, 45 instead of 39 on
// [3, 1021, 5, 80 / 48].)
//
// Measured, whole call: 594 us for [4, 4096, 16, 128] causal (1157 TFLOP/s of the
// formulas' five products, 1620 of the seven executed), 835 us for [1, 4096, 64,
// 192 / 128] with a shared key, 1404 us for [1, 32768, 2, 192 / 128].  The tensor
// pipe is active 76 % / 69 % of bwd_kernel on the first two: what bounds it is the
// chain of a tile (product, barrier, S or dP from tensor memory, exponential,
// P or dS back, barrier, product), which takes 2540 clocks per 128-query tile of
// the dK / dV pass where the products alone need 2048, and 1400 per 96-key tile of
// the dQ pass (products 1152), and at the change of items about 2900 clocks more.
// DRAM moves 545 + 184 MB in 568 us (dense_block).
template <int NCH, int NCV>
constexpr size_t smem_bytes() {
  const size_t nq = query_tile(NCH, NCV), nk = key_tile(NCH, NCV), own = (size_t)(NCH + NCV);
  const size_t kv = own * CH + query_stages(NCH, NCV) * (own * nq * 128 + 2 * nq * 4);
  const size_t q = own * CH + (kKeyStages * NCH + value_stages(NCH, NCV) * NCV) * nk * 128;
  return 1024 + 2 * kBarBytes + (kv > q ? kv : q);      // 1024: alignment
}

template <int NCH, int NCV, bool PACKED>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ Maps kv, const __grid_constant__ Maps qm,
               const __grid_constant__ Geo g) {
  static_assert(smem_bytes<NCH, NCV>() + 64 <= 227 * 1024, "shared memory");
  static_assert(64 * (NCH + NCV) + 2 * query_tile(NCH, NCV) + (p_apart(NCH, NCV) ? query_tile(NCH, NCV) / 2 : 0) <= 512 &&
                64 * NCH + 32 * q_in_tmem(NCH) + (do_in_tmem(NCH) ? 32 * NCV : 0) + 5 * key_tile(NCH, NCV) / 2 <= 512, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ volatile int abort_flag;
  __shared__ uint32_t tmem_slot;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform to the compiler
  if (threadIdx.x == 0) abort_flag = 0;
  if (warp == 1) { tmem_alloc(&tmem_slot, kTmemCols); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  await_previous();
  uint64_t *bars = reinterpret_cast<uint64_t*>(smem), *bars2 = bars + kBarBytes / 8;
  uint8_t* data = smem + 2 * kBarBytes;
  // one branch per role, its register share at the head of it: the compiler
  // allocates the code behind a setmaxnreg by that.  (A pass that gave up waiting
  // leaves the flag up: the second one ends at its first wait.)
  if (warp < 4) {
    regs_release<kRegsIssue>();
    dkv_pass<NCH, NCV, PACKED, kIssue>(p, kv, g, data, bars, tmem_base, abort_flag, warp, lane);
    dq_pass<NCH, NCV, PACKED, kIssue>(p, qm, g, data, bars2, tmem_base, abort_flag, warp, lane);
    if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
  } else if (warp < 8) {
    regs_release<kRegsOutput>();
    dkv_pass<NCH, NCV, PACKED, kOutput>(p, kv, g, data, bars, tmem_base, abort_flag, warp, lane);
    dq_pass<NCH, NCV, PACKED, kOutput>(p, qm, g, data, bars2, tmem_base, abort_flag, warp, lane);
  } else {
    regs_acquire<kRegsCompute>();
    dkv_pass<NCH, NCV, PACKED, kCompute>(p, kv, g, data, bars, tmem_base, abort_flag, warp, lane);
    dq_pass<NCH, NCV, PACKED, kCompute>(p, qm, g, data, bars2, tmem_base, abort_flag, warp, lane);
  }
}

// -------------------------------------------------------- short sequences
// Sequences of at most kAttnBwdShort positions: one block per (b, h) with q, k, v, do and
// o in shared memory as fp32 and fp32 arithmetic throughout (P and dS are not
// rounded).  A warp takes four queries, a lane a key of two of them, for P and dS;
// then a warp takes four rows of an output, a lane four of its columns.  The difference
// do . v - do . o is summed as do . (v - o), which is exact where a row has one key
// and o is its value: dq and dk of one-position sequences are exactly 0.
//
// Up to 16 positions this beats the tensor cores' 128-row tiles with few sequences
// and with many (us, against the kernels above; H = 16 or 4, d = 128): 8 of 4
// positions 8.2 (16.4), 8 of 16 10.2 (18.4), 8192 of 2 35 (309), of 8 94 (313), of
// 16 147 (315).  With 32 positions, eight warps and the same layout it lost with
// many: 545 (313).  Bound by the loads' latency with few, by shared-memory reads
// with many.
constexpr int kShortThreads = 128;       // at most: a warp per four rows, a thread per load while there are so many
constexpr int kShortPitch = 20;          // of P and dS: rows of 16-byte alignment
// Row pitch of `width` columns: whole 16 bytes, an odd number of them, so that 8
// lanes that read 16 bytes of 8 rows meet no bank twice.
__host__ __device__ constexpr int short_pitch(int width) { return 4 * (((width + 3) / 4) | 1); }

// Columns c .. c + 7 of a row of `width`, zeros behind it; and these as fp32 in
// shared memory, up to a multiple of four columns.
__device__ inline uint4 short_fetch(const __nv_bfloat16* row, int c, int width) {
  if (c + 8 <= width) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {};
#pragma unroll
  for (int y = 0; y < 7; ++y)
    if (c + y < width) w[y / 2] |= (uint32_t)__bfloat16_as_ushort(row[c + y]) << (16 * (y % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ inline void short_put(float* row, int c, int width, const uint4& w) {
  const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int y = 0; y < 2; ++y)
    if (c + 4 * y < width)
      *reinterpret_cast<float4*>(row + c + 4 * y) =
          make_float4(__uint_as_float(e[2 * y] << 16), __uint_as_float(e[2 * y] & 0xffff0000u),
                      __uint_as_float(e[2 * y + 1] << 16), __uint_as_float(e[2 * y + 1] & 0xffff0000u));
}
// a += x b for four columns
__device__ inline void short_add(float4& a, float x, const float4& b) {
  a.x = fmaf(x, b.x, a.x);
  a.y = fmaf(x, b.y, a.y);
  a.z = fmaf(x, b.z, a.z);
  a.w = fmaf(x, b.w, a.w);
}
// Columns c .. c + 3 of a row of `width`, times `scale`, as bf16; true if one is
// not finite as stored (the rounding to bf16 may take the largest to infinity).
__device__ inline bool short_store(__nv_bfloat16* row, int c, int width, const float4& v, float scale) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * scale, v.y * scale), hi = __floats2bfloat162_rn(v.z * scale, v.w * scale);
  if (c + 4 <= width) {
    *reinterpret_cast<uint2*>(row + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {                               // columns behind the row do not count
    if (c < width) row[c] = lo.x; else lo.x = zero.x;
    if (c + 1 < width) row[c + 1] = lo.y; else lo.y = zero.x;
    if (c + 2 < width) row[c + 2] = hi.x; else hi.x = zero.x;
    hi.y = zero.x;
  }
  const __nv_bfloat162 z = __hfma2(hi, zero, __hmul2(lo, zero));    // zeros, or NaN where a value is not finite
  return __low2float(z) != 0.f || __high2float(z) != 0.f;
}

__global__ void __launch_bounds__(kShortThreads, 4) short_kernel(const __grid_constant__ AttnBwdParams p) {
  extern __shared__ float4 short_smem[];
  await_previous();
  const int S = p.S, D = p.d_head + p.d_shared, pd = short_pitch(D), pv = short_pitch(p.d_v);
  float* q = reinterpret_cast<float*>(short_smem);
  float *k = q + S * pd, *v = k + S * pd, *dO = v + S * pv, *o = dO + S * pv, *P = o + S * pv, *dS = P + S * kShortPitch;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto at = [&](const void* base, const long long* st, int r) {
    return static_cast<const __nv_bfloat16*>(base) + b * st[0] + r * st[1] + h * st[2];
  };
  // every tensor's eight columns in flight before the first is stored
  const int n = (max(D, p.d_v) + 7) / 8;
  for (int x = threadIdx.x; x < S * n; x += blockDim.x) {
    const int r = x / n, c = 8 * (x - r * n);
    const bool own = c < p.d_head;
    uint4 wq = {}, wk = {}, wv = {}, wd = {}, wo = {};
    if (c < D) {
      wq = short_fetch(at(p.q, p.qs, r), c, D);
      wk = own ? short_fetch(at(p.k, p.kst, r), c, p.d_head)
               : short_fetch(static_cast<const __nv_bfloat16*>(p.ks) + b * p.kss[0] + r * p.kss[1], c - p.d_head, p.d_shared);
    }
    if (c < p.d_v) {
      wv = short_fetch(at(p.v, p.vs, r), c, p.d_v);
      wd = short_fetch(at(p.d_o, p.dos, r), c, p.d_v);
      wo = short_fetch(at(p.o, p.os, r), c, p.d_v);
    }
    short_put(q + r * pd, c, D, wq);
    short_put(k + r * pd, c, D, wk);
    short_put(v + r * pv, c, p.d_v, wv);
    short_put(dO + r * pv, c, p.d_v, wd);
    short_put(o + r * pv, c, p.d_v, wo);
  }
  __syncthreads();
  const int r0 = 4 * warp;               // this warp's four queries, then its four rows of each output
  int row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) row[r] = min(r0 + r, S - 1);
  if (r0 < S) {
    static_assert(kAttnBwdShort <= 16 && kAttnBwdShort <= kShortThreads / 8, "a half-warp holds the keys, the warps all rows");
    const int j = lane & 15, key = min(j, S - 1), i0 = r0 + 2 * (lane >> 4);
    const int query[2] = {min(i0, S - 1), min(i0 + 1, S - 1)};
    float s[2] = {}, x[2] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 a = *reinterpret_cast<const float4*>(k + key * pd + c);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 e = *reinterpret_cast<const float4*>(q + query[r] * pd + c);
        s[r] = fmaf(e.x, a.x, fmaf(e.y, a.y, fmaf(e.z, a.z, fmaf(e.w, a.w, s[r]))));
      }
    }
#pragma unroll 4
    for (int c = 0; c < p.d_v; c += 4) {
      const float4 a = *reinterpret_cast<const float4*>(v + key * pv + c);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 e = *reinterpret_cast<const float4*>(dO + query[r] * pv + c);
        const float4 m = *reinterpret_cast<const float4*>(o + query[r] * pv + c);
        x[r] = fmaf(e.x, a.x - m.x, fmaf(e.y, a.y - m.y, fmaf(e.z, a.z - m.z, fmaf(e.w, a.w - m.w, x[r]))));
      }
    }
    const float* lse = p.lse + (long long)blockIdx.x * S;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = i0 + r;
      if (i >= S) continue;
      const bool seen = j < S && (!p.causal || j <= i);
      const float e = expf(fmaf(p.scale, s[r], -lse[i]));
      P[i * kShortPitch + j] = seen ? e : 0.f;
      dS[i * kShortPitch + j] = seen ? e * x[r] : 0.f;
    }
  }
  __syncthreads();
  if (r0 >= S) return;
  bool bad = false;
  const int from = p.causal ? r0 : 0, to = p.causal ? min(S, r0 + 4) : S;   // queries of these keys, keys of these queries
  // rows r0 .. of M^T A (M: P or dS, A: rows of `pitch`), columns c .. c + 3
  auto keys = [&](const float* M, const float* A, int pitch, int c, float4 (&sum)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = from; i < S; ++i) {
      const float4 a = *reinterpret_cast<const float4*>(A + i * pitch + c), m = *reinterpret_cast<const float4*>(M + i * kShortPitch + r0);
      short_add(sum[0], m.x, a);
      short_add(sum[1], m.y, a);
      short_add(sum[2], m.z, a);
      short_add(sum[3], m.w, a);
    }
  };
  auto out = [&](void* base, const long long* st, int r) {
    return static_cast<__nv_bfloat16*>(base) + b * st[0] + (r0 + r) * st[1] + h * st[2];
  };
  for (int c = 4 * lane; c < p.d_v; c += 128) {
    float4 sum[4];
    keys(P, dO, pv, c, sum);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r0 + r < S) bad |= short_store(out(p.dv, p.dvs, r), c, p.d_v, sum[r], 1.f);
  }
  const int pitch = part_pitch(p.d_shared);
  for (int c = 4 * lane; c < D; c += 128) {
    float4 sum[4];
    keys(dS, q, pd, c, sum);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r0 + r >= S) continue;
      if (c < p.d_head) {
        bad |= short_store(out(p.dk, p.dks, r), c, p.d_head, sum[r], p.scale);
      } else {
        const float4 w = make_float4(sum[r].x * p.scale, sum[r].y * p.scale, sum[r].z * p.scale, sum[r].w * p.scale);
        const float z = fmaf(w.x, 0.f, fmaf(w.y, 0.f, fmaf(w.z, 0.f, w.w * 0.f)));
        *reinterpret_cast<float4*>(p.part + ((long long)blockIdx.x * S + r0 + r) * pitch + c - p.d_head) = w;
        bad |= z != z;
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = 0; j < to; ++j) {
      const float4 a = *reinterpret_cast<const float4*>(k + j * pd + c);
#pragma unroll
      for (int r = 0; r < 4; ++r) short_add(sum[r], dS[row[r] * kShortPitch + j], a);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r0 + r < S) bad |= short_store(out(p.dq, p.dqs, r), c, D, sum[r], p.scale);
  }
  if (bad) set_status(p.status, MC_STATUS_NONFINITE_UPDATE);
}

// ------------------------------------------------------------- shared key
// dk_shared[b, j, c] = sum over the heads, in order, of the fp32 partial sums
// [b][h][j][c] (rows of part_pitch values).  A thread takes four features of a
// position, eight heads' loads in flight.  15.2 us for the 67 MB of k2_mla_layer
// (16.4 in blocks of 256 threads, one or two per SM).
constexpr int kSharedThreads = 64;
__global__ void __launch_bounds__(kSharedThreads) shared_kernel(const __grid_constant__ AttnBwdParams p, const int blocks) {
  const int quads = part_pitch(p.d_shared) / 4, b = blockIdx.x / blocks;
  await_previous();
  const long long per = (long long)p.S * quads, e = (long long)(blockIdx.x - b * blocks) * kSharedThreads + threadIdx.x;
  if (e >= per) return;
  const float4* src = reinterpret_cast<const float4*>(p.part) + (long long)b * p.H * per + e;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& v) { s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w; };
  int h = 0;
  for (; h + 8 <= p.H; h += 8) {
    float4 v[8];
#pragma unroll
    for (int y = 0; y < 8; ++y) v[y] = src[(h + y) * per];
#pragma unroll
    for (int y = 0; y < 8; ++y) add(v[y]);
  }
  for (; h < p.H; ++h) add(src[h * per]);
  const int j = (int)(e / quads), c = 4 * (int)(e - (long long)j * quads);
  __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.dksh) + b * p.dkshs[0] + j * p.dkshs[1];
  // finite parts may have a sum that is not
  if (short_store(to, c, p.d_shared, s, 1.f)) set_status(p.status, MC_STATUS_NONFINITE_UPDATE);
}

// dK and dV of the key blocks whose query tiles were divided among items (span_of in
// dkv_pass), the parts added up in their order: a block of threads per kJoinRows keys of a
// head, few enough that all of a thread's loads are in flight at once.
constexpr int kJoinThreads = 256, kJoinRows = 16;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ Geo g) {
  await_previous();
  const int heads = p.H / g.q_heads, b = blockIdx.x / (BM / kJoinRows), r0 = (blockIdx.x - b * (BM / kJoinRows)) * kJoinRows;
  const int e = b / heads, h = b - e * heads;
  if (e >= *g.count) return;
  const int4 blk = *reinterpret_cast<const int4*>(g.blocks + e);         // start, length, index
  if (blk.x < 0 || blk.y < 1 || blk.x > p.S - blk.y || blk.z < 0 || blk.z > (blk.y - 1) / BM) return;
  const int tiles = ((blk.y + BM - 1) / BM - blk.z) * g.q_heads, per = max((tiles + g.parts - 1) / g.parts, kPartTiles);
  const int parts = (tiles + per - 1) / per;
  if (parts < 2) return;
  const int pitch = packed_part_pitch(p.d_head, p.d_v), quads = pitch / 4, of_v = part_pitch(p.d_v);
  const int rows = min(kJoinRows, blk.y - blk.z * BM - r0);
  const long long first = blk.x + blk.z * BM + r0;
  bool bad = false;
#pragma unroll 4
  for (int i = threadIdx.x; i < rows * quads; i += kJoinThreads) {
    const int r = i / quads, c = 4 * (i - r * quads);
    const long long row = first + r;
    const float4* src = reinterpret_cast<const float4*>(p.part + ((long long)h * g.parts * p.S + row) * pitch + c);
    float4 s = src[0];
#pragma unroll 4
    for (int k = 1; k < parts; ++k) {
      const float4 v = src[(long long)k * p.S * quads];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const bool is_v = c < of_v;
    __nv_bfloat16* to = is_v ? static_cast<__nv_bfloat16*>(p.dv) + row * p.dvs[1] + h * p.dvs[2]
                             : static_cast<__nv_bfloat16*>(p.dk) + row * p.dks[1] + h * p.dks[2];
    bad |= short_store(to, is_v ? c : c - of_v, is_v ? p.d_v : p.d_head, s, 1.f);
  }
  if (bad) set_status(p.status, MC_STATUS_NONFINITE_UPDATE);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode() {
  static EncodeTiledFn fn = [] {
    cudaDriverEntryPointQueryResult qr;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(f);
    return static_cast<EncodeTiledFn>(nullptr);
  }();
  return fn;
}

// [B, S, H, width] (or [B, S, width] with H = 0) in boxes of 64 features x `rows`
bool encode(CUtensorMap* m, const void* base, int width, int H, int S, int B, const long long* st, int rows) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const int rank = H ? 4 : 3;
  cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t by[3] = {(cuuint64_t)(H ? st[2] : 0) * 2, (cuuint64_t)st[1] * 2, (cuuint64_t)st[0] * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1}, es[4] = {1, 1, 1, 1};
  if (!H) {
    dims[1] = (cuuint64_t)S; dims[2] = (cuuint64_t)B;
    by[0] = (cuuint64_t)st[1] * 2; by[1] = (cuuint64_t)st[0] * 2;
    box[1] = (cuuint32_t)rows; box[2] = 1;
  }
  return encode_bound([&] {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, by, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

bool geometry(const AttnBwdParams& p, Geo& g, char* err, size_t errlen) {
  g.nck = (p.d_head + 63) / 64;
  g.nch = p.d_shared > 0 ? g.nck + (p.d_shared + 63) / 64 : g.nck;
  g.ncv = (p.d_v + 63) / 64;
  g.nb = (p.S + BM - 1) / BM;
  g.nt = (p.S + query_tile(g.nch, g.ncv) - 1) / query_tile(g.nch, g.ncv);
  const long long items = (long long)p.B * p.H * g.nb;
  if (items >= (1ll << 30)) { snprintf(err, errlen, "%lld work items exceed the kernel's 2^30", items); return false; }
  g.items = (int)items;
  g.heads = p.B * p.H;
  g.group = 512 / g.nb < 1 ? 1 : 512 / g.nb;
  if (g.group > g.heads) g.group = g.heads;
  g.full = g.heads / g.group * g.group * g.nb;
  g.sp = attn_bwd_padded_rows(p.S);
  g.div_group_items = make_fastdiv((uint32_t)(g.group * g.nb));
  g.div_group = make_fastdiv((uint32_t)g.group);
  g.div_last = make_fastdiv((uint32_t)(g.heads % g.group ? g.heads % g.group : 1));
  g.div_h = make_fastdiv((uint32_t)p.H);
  return true;
}

template <int NCH, int NCV, bool PACKED>
cudaError_t launch_passes(const AttnBwdParams& p, const Maps& kv, const Maps& qm, const Geo& g, int grid, cudaStream_t s) {
  constexpr size_t smem = smem_bytes<NCH, NCV>();
  const cudaError_t e = cudaFuncSetAttribute(bwd_kernel<NCH, NCV, PACKED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_behind(bwd_kernel<NCH, NCV, PACKED>, (unsigned)grid, kThreads, smem, s, p, kv, qm, g);
}

}  // namespace ab
}  // namespace

// Rows of nlse and delta per (b, h): whole 128-row blocks and whole 96-row
// tiles both end inside.
long long attn_bwd_padded_rows(int S) {
  const long long a = round_up(S, 128), b = round_up(S, 96);
  return round_up(a > b ? a : b, 32);
}

bool attn_bwd_supported(const AttnBwdParams& p, char* err, size_t errlen) {
  const int D = p.d_head + p.d_shared;
  if (D < 16 || D > 192) { snprintf(err, errlen, "q.k length %d outside [16, 192]", D); return false; }
  if (p.d_v < 16 || p.d_v > 128) { snprintf(err, errlen, "d_v %d outside [16, 128]", p.d_v); return false; }
  if (p.d_shared > 0 && (p.d_head % 64) != 0) {
    snprintf(err, errlen, "with a shared key part d_head must be a multiple of 64 (got %d)", p.d_head);
    return false;
  }
  ab::Geo g;
  return ab::geometry(p, g, err, errlen);
}

cudaError_t launch_attn_bwd(const AttnBwdParams& p, cudaStream_t s, char* err, size_t errlen) {
  using namespace ab;
  Geo g;
  if (!geometry(p, g, err, errlen)) return cudaErrorInvalidValue;
  auto sum_heads = [&]() -> cudaError_t {
    if (p.d_shared == 0) return cudaSuccess;
    const long long blocks = cdiv((long long)p.S * (part_pitch(p.d_shared) / 4), kSharedThreads);
    if (blocks * p.B > 0x7fffffff) { snprintf(err, errlen, "too many rows for one launch"); return cudaErrorInvalidValue; }
    return launch_behind(shared_kernel, (unsigned)(blocks * p.B), kSharedThreads, 0, s, p, (int)blocks);
  };
  if (p.S <= kAttnBwdShort) {
    const int pd = short_pitch(p.d_head + p.d_shared), pv = short_pitch(p.d_v);
    const size_t smem = (size_t)p.S * (2 * pd + 3 * pv + 2 * kShortPitch) * 4;
    // the limit belongs to the kernel, not to this call: always that of the largest,
    // so that another thread's call cannot lower it before this launch
    constexpr int most = kAttnBwdShort * (2 * short_pitch(192) + 3 * short_pitch(128) + 2 * kShortPitch) * 4;
    cudaError_t e = cudaFuncSetAttribute(short_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    const int width = p.d_head + p.d_shared > p.d_v ? p.d_head + p.d_shared : p.d_v;
    const int want = p.S * (width > 64 ? (width + 7) / 8 : 8);       // 8 S: a warp per four rows
    const int threads = want < kShortThreads ? (want + 31) / 32 * 32 : kShortThreads;
    e = launch_behind(short_kernel, (unsigned)g.heads, (unsigned)threads, smem, s, p);
    return e != cudaSuccess ? e : sum_heads();
  }
  const int nq = query_tile(g.nch, g.ncv), D = p.d_head + p.d_shared;
  const int nk = key_tile(g.nch, g.ncv);
  Maps kv, qm;                            // for dkv (128-row keys, nq-row queries) and dq (nk-row keys, 128-row queries)
  memset(&kv, 0, sizeof kv);
  bool ok = encode(&kv.q, p.q, D, p.H, p.S, p.B, p.qs, nq) && encode(&kv.k, p.k, p.d_head, p.H, p.S, p.B, p.kst, BM) &&
            encode(&kv.v, p.v, p.d_v, p.H, p.S, p.B, p.vs, BM) && encode(&kv.d_o, p.d_o, p.d_v, p.H, p.S, p.B, p.dos, nq) &&
            (p.d_shared == 0 || encode(&kv.ks, p.ks, p.d_shared, 0, p.S, p.B, p.kss, BM));
  qm = kv;
  if (nq != BM)
    ok = ok && encode(&qm.q, p.q, D, p.H, p.S, p.B, p.qs, BM) && encode(&qm.d_o, p.d_o, p.d_v, p.H, p.S, p.B, p.dos, BM);
  if (nk != BM)
    ok = ok && encode(&qm.k, p.k, p.d_head, p.H, p.S, p.B, p.kst, nk) && encode(&qm.v, p.v, p.d_v, p.H, p.S, p.B, p.vs, nk) &&
         (p.d_shared == 0 || encode(&qm.ks, p.ks, p.d_shared, 0, p.S, p.B, p.kss, nk));
  if (!ok) { snprintf(err, errlen, "tensor map encoding failed"); return cudaErrorInvalidValue; }
  const int sms = sm_count();
  const long long ni = cdiv(g.sp, kRowPos), nh = cdiv(p.H, kRowHeads);
  if (ni * nh * p.B > 0x7fffffff) { snprintf(err, errlen, "too many rows for one launch"); return cudaErrorInvalidValue; }
  cudaError_t e = launch_behind(rows_kernel<false>, (unsigned)(ni * nh * p.B), 256, 0, s, p, (int)g.sp, (int)ni, (int)nh, nullptr, nullptr);
  if (e != cudaSuccess) return e;
  const int grid = 2 * g.items < sms ? 2 * g.items : sms;
  using Launch = cudaError_t (*)(const AttnBwdParams&, const Maps&, const Maps&, const Geo&, int, cudaStream_t);
  static const Launch by_chunks[3][2] = {{launch_passes<1, 1, false>, launch_passes<1, 2, false>},
                                         {launch_passes<2, 1, false>, launch_passes<2, 2, false>},
                                         {launch_passes<3, 1, false>, launch_passes<3, 2, false>}};
  e = by_chunks[g.nch - 1][g.ncv - 1](p, kv, qm, g, grid, s);
  return e != cudaSuccess ? e : sum_heads();
}

// Packed sequences: the dense passes' parameters with one batch, token strides, and
// the plan's list in the place of the order of blocks.
cudaError_t launch_packed_bwd(const PackedBwdParams& a, int blocks, cudaStream_t s, char* err, size_t errlen) {
  using namespace ab;
  AttnBwdParams p;
  Geo g;
  memset(&p, 0, sizeof p);
  memset(&g, 0, sizeof g);
  p.B = 1; p.S = a.T; p.H = a.H; p.d_head = a.d; p.d_v = a.d_v;
  p.causal = 1;
  p.scale = a.scale;
  p.q = a.q; p.k = a.k; p.v = a.v; p.o = a.o; p.d_o = a.d_o;
  p.lse = a.lse;
  p.dq = a.dq; p.dk = a.dk; p.dv = a.dv;
  for (int i = 0; i < 2; ++i) {
    p.os[i + 1] = a.os[i]; p.dos[i + 1] = a.dos[i];
    p.dqs[i + 1] = a.dqs[i]; p.dks[i + 1] = a.dks[i]; p.dvs[i + 1] = a.dvs[i];
  }
  p.nlse = a.nlse; p.ndelta = a.ndelta;
  p.counter = a.counter;
  p.status = a.status;
  g.nch = g.nck = (a.d + 63) / 64;
  g.ncv = (a.d_v + 63) / 64;
  g.sp = a.padded;
  g.q_heads = a.group;
  g.parts = a.parts;
  p.part = a.part;
  g.order[0] = a.by_key_head;
  g.order[1] = a.by_head;
  g.blocks = a.blocks;
  g.count = a.count;
  g.fill = a.fill;
  const int nq = query_tile(g.nch, g.ncv), nk = key_tile(g.nch, g.ncv), Hkv = a.H / a.group;
  static_assert(query_tile(2, 2) == BM, "the padded rows end with whole blocks of 128");
  Maps kv, qm;
  memset(&kv, 0, sizeof kv);
  auto encode = [&](CUtensorMap* m, const void* base, int width, int heads, const long long* st, int rows) {
    return packed::encode_rows(m, base, width, heads, a.T, st, rows);
  };
  bool ok = encode(&kv.q, a.q, a.d, a.H, a.qs, nq) && encode(&kv.d_o, a.d_o, a.d_v, a.H, a.dos, nq) &&
            encode(&kv.k, a.k, a.d, Hkv, a.ks, BM) && encode(&kv.v, a.v, a.d_v, Hkv, a.vs, BM);
  qm = kv;
  if (nk != BM) ok = ok && encode(&qm.k, a.k, a.d, Hkv, a.ks, nk) && encode(&qm.v, a.v, a.d_v, Hkv, a.vs, nk);
  if (!ok) { snprintf(err, errlen, "tensor map encoding failed"); return cudaErrorInvalidValue; }
  const long long ni = (long long)blocks * (BM / kRowPos), nh = cdiv(a.H, kRowHeads);
  if (ni * nh > 0x7fffffff) { snprintf(err, errlen, "too many rows for one launch"); return cudaErrorInvalidValue; }
  const cudaError_t e = launch_behind(rows_kernel<true>, (unsigned)(ni * nh), 256, 0, s, p, (int)g.sp, (int)ni, (int)nh, a.blocks, a.count);
  if (e != cudaSuccess) return e;
  const long long items = (long long)blocks * (a.H + Hkv * a.parts);
  const int grid = items < sm_count() ? (int)items : sm_count();
  using Launch = cudaError_t (*)(const AttnBwdParams&, const Maps&, const Maps&, const Geo&, int, cudaStream_t);
  static const Launch by_chunks[2][2] = {{launch_passes<1, 1, true>, launch_passes<1, 2, true>},
                                         {launch_passes<2, 1, true>, launch_passes<2, 2, true>}};
  const cudaError_t passes = by_chunks[g.nch - 1][g.ncv - 1](p, kv, qm, g, grid, s);
  if (passes != cudaSuccess || a.parts == 1) return passes;
  return launch_behind(join_kernel, (unsigned)(blocks * Hkv * (BM / kJoinRows)), kJoinThreads, 0, s, p, g);
}

}  // namespace mc
