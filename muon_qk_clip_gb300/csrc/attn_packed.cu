// Causal attention over packed sequences with grouped heads, and the per-head max
// logit on the way ([K2-internals] "核心数学": O^h = softmax(scale Q^h K^h^T) V^h,
// S_max^h over every sequence).  T tokens hold the sequences one behind the other,
// sequence s from offsets[s] to offsets[s + 1]; query head h reads key and value
// head h / (H / H_kv); a token sees the tokens of its own sequence up to itself.
//
//   plan_kernel   one block: the sequences' bounds from `offsets`, and their blocks
//                 of query rows in a list, those with most keys first
//   fwd_kernel    persistent, one CTA per SM; an item is two 128-row query tiles
//                 that share their keys and values: the same rows of two heads of a
//                 group, or (groups of an odd number of heads, unless their sequences
//                 are short) 256 rows of one head
//
// Warps of fwd_kernel: 0 producer (TMA), 1 MMA issuer, 2 and 3 rows of no sequence, 4..7 output, 8..11 and
// 12..15 softmax of the two tiles, a thread per query row.  Tensor memory: S of
// both tiles (128 columns each; P, in bf16, over its first half) and O of both.
// Per key block j the tensor core gets, tile by tile, O += P(j) V(j) and S(j + 1) =
// Q K(j + 1)^T: while it works for one tile, the other's softmax warps turn S into P.
// S(j + 1) overwrites P(j) behind O's reads of it without a wait: the tensor core
// executes the products that one thread issues in their order (as seen on this
// hardware; the dense backward rests on the same).
//
// Bound by each tile's chain, scores to P, of which the two tiles overlap only a part:
// 16384 tokens in eight documents, 32 / 8 heads of 128, 300 us at first and 320 in a long
// run of calls, under the power limit, 1.27 and 1.19 PFLOP/s; 24571 in one, 16 / 2 heads,
// 1500 and 1600 us, 1.65 and 1.54 (measured peak 1.93; the tensor pipe is 67 % active, the
// exponentials' a third).  Beyond the long one's rate the documents take some 4 us for each
// of an SM's 14 items (as a whole; its parts are not measured).  The first scores of the
// next item behind the last products of one (323 to 321 us in one run), P handed over in halves (319; the long one 1648 to
// 1605), finite checks on the diagonal's blocks alone and these by groups of 32
// columns (307; 1550) were kept in that order.
//
// The running maximum is updated lazily, when a block's maximum exceeds it by more
// than 8 in log2: O and the row sum are then rescaled by the softmax warps, behind
// the S that they wait for anyway, whose completion means O's too.  P <= 2^8, and
// the result is exact either way.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.h"
#include "packed.cuh"

namespace mc {
namespace {
namespace pf {
using namespace attn;
using namespace packed;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;

// ------------------------------------------------------------------- plan
// Blocks of `rows` rows of every sequence, sorted by descending index in their
// sequence (a causal block's work grows with it).  A sequence of n blocks has one
// block of each index below n, so the place of the blocks of index c is the number
// of those above it: with cnt(c) = sequences that have more than c blocks, the sum
// of cnt over c' > c; sequences take the places within it as they come (their order
// changes nothing but the schedule).
//
// Offsets are data on the device: a value below its predecessor or beyond T is
// taken as its predecessor or T, which keeps every access inside and every
// sequence apart, and sets MC_STATUS_BAD_OFFSETS.
//
// The lists that only the plan reads stay in shared memory where they fit (prompts
// of 366 tokens in all: 5 us alone, 7 with the lists in the workspace, whose
// searches are chains of dependent loads).
constexpr int kPlanThreads = 1024;
constexpr size_t kPlanLocal = 46 * 1024;

// Inclusive scan over the block; `carry` is the value before its first thread, and
// becomes that of its last.
template <bool MAX>
__device__ inline int block_scan(int v, int* warps, int& carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto op = [](int a, int b) { return MAX ? max(a, b) : a + b; };
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = op(u, v);
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = op(u, w);
    }
    warps[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v = op(warps[warp - 1], v);
  v = op(carry, v);
  carry = op(carry, warps[31]);
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PackedPlan p) {
  __shared__ int warps[32];
  __shared__ int most;
  extern __shared__ int local[];
  int* bounds = p.local ? local : p.bounds;
  int* first = p.local ? bounds + p.nseq + 1 : p.first;
  int* place = p.local ? first + p.nseq : p.place;
  await_previous();
  release_next();
  const int tid = threadIdx.x;
  if (tid == 0) most = 0;
  if (tid < 2) p.counter[tid] = 0;
  if (p.smax)
    for (int h = tid; h < p.H; h += kPlanThreads) p.smax[h] = -INFINITY;
  // bounds[s]: offsets made monotone within [0, T]
  int carry = 0;
  bool bad = false;
  for (int s0 = 0; s0 <= p.nseq; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int v = s <= p.nseq ? p.offsets[s] : 0, c = block_scan<true>(min(max(v, 0), p.T), warps, carry);
    if (s <= p.nseq) {
      bounds[s] = c;
      bad |= c != v;
    }
  }
  if (bad) set_status(p.status, MC_STATUS_BAD_OFFSETS);
  if (tid == 0) p.count[2] = carry;      // the last offset, made monotone
  // first[s]: blocks of the sequences before s; place[n]: sequences of n blocks
  for (int c = tid; c <= p.capacity; c += kPlanThreads) place[c] = 0;
  __syncthreads();
  carry = 0;
  int my_most = 0;
  for (int s0 = 0; s0 < p.nseq; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const int n = s < p.nseq ? (bounds[s + 1] - bounds[s] + p.rows - 1) / p.rows : 0;
    const int end = block_scan<false>(n, warps, carry);
    if (s < p.nseq) first[s] = end - n;
    if (n > 0) atomicAdd(&place[n], 1);
    my_most = max(my_most, n);
  }
  const int total = carry;
  if (my_most > 0) atomicMax(&most, my_most);
  __syncthreads();
  // place[c], c = number of a block counted from 1: blocks with a larger number
  int above = 0, before = 0;             // sequences of more blocks; blocks of larger numbers
  for (int c0 = most; c0 > 0; c0 -= kPlanThreads) {
    const int c = c0 - tid;
    const int cnt = block_scan<false>(c > 0 ? place[c] : 0, warps, above);    // sequences of at least c blocks
    const int upto = block_scan<false>(c > 0 ? cnt : 0, warps, before);
    __syncthreads();
    if (c > 0) place[c] = upto - cnt;
  }
  __syncthreads();
  for (int x = tid; x < total; x += kPlanThreads) {
    int lo = 0, hi = p.nseq;             // the last sequence whose first block is at or before x, and has blocks
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= x) lo = mid; else hi = mid;
    }
    const int b = x - first[lo], start = bounds[lo];
    p.blocks[atomicAdd(&place[b + 1], 1)] = make_int4(start, bounds[lo + 1] - start, b, packed_pad(start, lo));
  }
  if (tid == 0) {
    *p.count = total;
    p.count[1] = bounds[0];
  }
}

// ---------------------------------------------------------------- forward
constexpr int BM = 128, CH = BM * 128;   // rows of a tile; bytes of one 64-feature chunk (128-byte swizzle)
constexpr int kThreads = 512;
// The launch's 128 registers a thread dealt out again per group of four warps: the
// sum over the groups, 72 + 72 + 184 + 184, is the launch's 4 x 128.
constexpr int kRegsIssue = 72, kRegsOutput = 72, kRegsSoftmax = 184;
constexpr uint32_t kTmemCols = 512, kO = 256;
constexpr int kBarBytes = 512;

__host__ __device__ constexpr int stage_bytes(int nch, int ncv) { return (nch > ncv ? nch : ncv) * CH; }
__host__ __device__ constexpr int stages(int nch, int ncv) { return nch > 1 || ncv > 1 ? 4 : 6; }
__host__ __device__ constexpr size_t smem_bytes(int nch, int ncv) {
  return 1024 + 2 * (size_t)nch * CH + (size_t)stages(nch, ncv) * stage_bytes(nch, ncv) + 2 * BM * 4 + kBarBytes;
}

struct Maps {
  CUtensorMap q, k, v;
};

__device__ inline void block_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ inline float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// First row, key blocks and head of tile t of an item.
struct Tile {
  int row0, nkv, head;
};
__device__ inline Tile tile_of(const PackedFwdParams& p, const Item& x, int t) {
  Tile r;
  r.row0 = p.pairs ? x.b.index * BM : (2 * x.b.index + t) * BM;
  r.head = x.head;
  bool there = r.row0 < x.b.len;
  if (p.pairs) {                         // the last pair of a group of an odd number has one head
    const int key = x.head / p.pairs, at = 2 * (x.head - key * p.pairs) + t;
    r.head = key * p.group + at;
    there = there && at < p.group;
  }
  r.nkv = there ? r.row0 / BM + 1 : 0;
  return r;
}

enum Role { kIssue, kOutput, kSoftmax };

template <int NCH, int NCV, int ROLE>
__device__ __forceinline__ void forward(const PackedFwdParams& p, const Maps& mp, uint8_t* smem, uint32_t tmem, volatile int& abort_flag,
                                        int warp, int lane) {
  constexpr int kStages = stages(NCH, NCV), kStageBytes = stage_bytes(NCH, NCV);
  uint8_t* qbuf = smem;                                  // two tiles x NCH chunks
  uint8_t* kvbuf = qbuf + 2 * NCH * CH;                  // stages: keys and values in turn
  float* inv = reinterpret_cast<float*>(kvbuf + kStages * kStageBytes);       // [2][BM] 1 / row sum
  uint64_t* bars = reinterpret_cast<uint64_t*>(inv + 2 * BM);
  uint64_t* q_full = bars + 0;       // [2] tiles
  uint64_t* q_empty = bars + 2;      // [2]
  uint64_t* s_full = bars + 4;       // [2]
  uint64_t* p_full = bars + 6;       // [2] 4 warps: all of P
  uint64_t* o_full = bars + 8;       // [2]
  uint64_t* o_empty = bars + 10;     // [2] 4 warps: O and the row sums have been read
  uint64_t* l_full = bars + 12;      // [2] 4 warps: row sums
  uint64_t* drain = bars + 14;
  uint64_t* kv_full = bars + 15;     // [stages <= 6]
  uint64_t* kv_empty = bars + 21;    // [6]
  uint64_t* p_half = bars + 35;      // [2] 4 warps: the first 64 keys of P
  const Ring ring = {reinterpret_cast<volatile int*>(bars + 38), bars + 27, bars + 31};
  static_assert(38 * 8 + kRing * kSlot * 4 <= kBarBytes, "barriers");
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1); mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1); mbar_init(&p_full[t], 4); mbar_init(&p_half[t], 4);
      mbar_init(&o_full[t], 1); mbar_init(&o_empty[t], 4);
      mbar_init(&l_full[t], 4);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < kStages; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int s = 0; s < kRing; ++s) { mbar_init(&ring.full[s], 1); mbar_init(&ring.empty[s], 13); }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) { prefetch_tmap(&mp.q); prefetch_tmap(&mp.k); prefetch_tmap(&mp.v); }
  block_sync();
  auto fail = [&]() { abort_flag = 1; set_status(p.status, MC_STATUS_TIMEOUT); };

  if (ROLE == kIssue && warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const int count = *p.count, rows = p.pairs ? BM : 2 * BM;
      uint32_t s = 0, ph = 0, nq[2] = {0, 0};
      uint32_t used_q = 0, par_q[2] = {}, used_kv = 0, par_kv = 0;      // bits: stages used, and their last phase
      auto load_q = [&](const Item& x, int t) -> bool {
        const Tile tl = tile_of(p, x, t);
        if (!mbar_wait(&q_empty[t], (nq[t] & 1) ^ 1, &abort_flag)) return false;
        mbar_arrive_expect_tx(&q_full[t], NCH * CH);
        for (int c = 0; c < NCH; ++c) load_rows<BM>(qbuf + (t * NCH + c) * CH, &mp.q, &q_full[t], c, tl.head, x.b, tl.row0);
        used_q |= 1u << t;
        par_q[t] = nq[t]++ & 1;
        return true;
      };
      auto load_kv = [&](const Item& x, const CUtensorMap* map, int chunks, int head, int j) -> bool {
        if (!mbar_wait(&kv_empty[s], ph ^ 1, &abort_flag)) return false;
        mbar_arrive_expect_tx(&kv_full[s], chunks * CH);
        for (int c = 0; c < chunks; ++c) load_rows<BM>(kvbuf + s * kStageBytes + c * CH, map, &kv_full[s], c, head, x.b, j * BM);
        used_kv |= 1u << s;
        par_kv = (par_kv & ~(1u << s)) | ph << s;
        if (++s == kStages) { s = 0; ph ^= 1; }
        return true;
      };
      int next = atomicAdd(p.counter, 1);
      Item x = item_at(p.blocks, count, p.order, p.T, rows, next), y = x;
      bool ok = ring_put(ring, 0, x, &abort_flag);
      for (uint32_t n = 1; ok && x.head >= 0; x = y, ++n) {
        const Tile t0 = tile_of(p, x, 0), t1 = tile_of(p, x, 1);
        const int nkv = max(t0.nkv, t1.nkv), head = t0.head / p.group;
        ok = load_q(x, 0);
        for (int j = 0; ok && j < nkv; ++j) {
          if (j == max(0, nkv - 2)) next = atomicAdd(p.counter, 1);
          if (j == nkv - 1) {
            y = item_at(p.blocks, count, p.order, p.T, rows, next);
            if (!ring_put(ring, n, y, &abort_flag)) { ok = false; break; }
          }
          ok = load_kv(x, &mp.k, NCH, head, j) && (j > 0 || t1.nkv == 0 || load_q(x, 1)) && load_kv(x, &mp.v, NCV, head, j);
        }
      }
      if (!ok) fail();
      // every issued copy must have landed before the CTA may exit
      for (int t = 0; t < 2; ++t)
        if (used_q >> t & 1) mbar_wait(&q_full[t], par_q[t], nullptr);
      for (int i = 0; i < kStages; ++i)
        if (used_kv >> i & 1) mbar_wait(&kv_full[i], par_kv >> i & 1, nullptr);
    }
  } else if (ROLE == kIssue && warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = make_idesc_bf16(BM, BM, 0, 0);          // Q x K, both K-major
    constexpr uint32_t idesc_o = make_idesc_bf16(BM, 64 * NCV, 0, 1);    // P (tensor memory) x V (MN-major)
    const uint64_t dq_ = make_sdesc_sw128(smem_u32(qbuf), 16, 1024), dk_ = make_sdesc_sw128(smem_u32(kvbuf), 16, 1024);
    const uint64_t dv_ = make_sdesc(smem_u32(kvbuf), CH, 1024, 2);
    uint32_t s = 0, ph = 0, nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};
    bool issued = false, ok = true;
    auto scores = [&](int t, uint32_t stage, bool last) {     // S of tile t from the keys in `stage`; `last`: its Q is free after it
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4 * NCH; ++c)
          tc_mma(tmem + t * BM, dq_ + (t * NCH * CH + (c >> 2) * CH + (c & 3) * 32) / 16,
                 dk_ + (stage * kStageBytes + (c >> 2) * CH + (c & 3) * 32) / 16, idesc_s, c > 0);
        tc_commit(&s_full[t]);
        if (last) tc_commit(&q_empty[t]);
      }
      __syncwarp();
    };
    auto done = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    auto weighted = [&](int t, uint32_t stage, int half, bool add) {     // O of tile t (+)= P V for 64 keys
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BM / 32; ++kk)
          tc_mma_ts(tmem + kO + t * BM, tmem + t * BM + (half * BM / 32 + kk) * 8,
                    dv_ + (stage * kStageBytes) / 16 + (half * BM / 32 + kk) * 128, idesc_o, (add || kk > 0) ? 1u : 0u);
      }
      __syncwarp();
    };
    // first scores of an item's tile t from the keys in `stage`
    auto begin = [&](int t, uint32_t stage, int blocks) -> bool {
      if (!warp_wait(&q_full[t], nq[t]++ & 1, &abort_flag)) return false;
      tc_fence_after();
      scores(t, stage, blocks == 1);
      return true;
    };
    Item x;
    int n[2] = {0, 0};                   // key blocks of the item's tiles
    auto next_item = [&](uint32_t li) -> bool {
      if (!ring_get(ring, li, x, &abort_flag)) return false;
      n[0] = x.head < 0 ? 0 : tile_of(p, x, 0).nkv;
      n[1] = x.head < 0 ? 0 : tile_of(p, x, 1).nkv;
      return true;
    };
    ok = next_item(0);
    if (ok && n[0] > 0) {
      ok = warp_wait(&kv_full[s], ph, &abort_flag) && begin(0, s, n[0]) && (n[1] == 0 || begin(1, s, n[1]));
      issued = true;
      done(&kv_empty[s]);
      if (++s == kStages) { s = 0; ph ^= 1; }
    }
    for (uint32_t li = 1; ok && n[0] > 0; ++li) {
      const int cur[2] = {n[0], n[1]}, nkv = max(n[0], n[1]);
      for (int j = 0; j < nkv && ok; ++j) {
        const uint32_t sv = s;
        if (!(ok = warp_wait(&kv_full[sv], ph, &abort_flag))) break;
        if (++s == kStages) { s = 0; ph ^= 1; }
        // behind an item's last products come the next item's first scores, tile by tile,
        // so that the two tiles' softmax stay half a period apart
        const bool last = j + 1 == nkv;
        if (last && !(ok = next_item(li))) break;
        const bool more = !last || n[0] > 0;
        if (more && !(ok = warp_wait(&kv_full[s], ph, &abort_flag))) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j < cur[t]) {
            // the first half of P's keys is multiplied while the second is in the making
            if (!(ok = warp_wait(&p_half[t], np[t] & 1, &abort_flag))) break;
            if (j == 0 && !(ok = warp_wait(&o_empty[t], (no[t]++ & 1) ^ 1, &abort_flag))) break;
            tc_fence_after();
            weighted(t, sv, 0, j > 0);
            if (!(ok = warp_wait(&p_full[t], np[t]++ & 1, &abort_flag))) break;
            tc_fence_after();
            weighted(t, sv, 1, true);
            if (j + 1 == cur[t]) done(&o_full[t]);
            if (j + 1 < cur[t]) scores(t, s, j + 2 == cur[t]);
          }
          if (last && n[t] > 0 && !(ok = begin(t, s, n[t]))) break;
        }
        if (!ok) break;
        done(&kv_empty[sv]);
        if (more) {
          done(&kv_empty[s]);
          if (++s == kStages) { s = 0; ph ^= 1; }
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (issued) {
      done(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else if (ROLE == kIssue) {
    // ------------------------------------------------------------ rows of no sequence
    const Outside out = outside_of(p.count, p.T);
    const int w = 2 * blockIdx.x + warp - 2, warps = 2 * gridDim.x;
    if (p.fill & MC_FILL_O) fill_rows(out, p.o, p.os, p.H, p.d_v, w, warps);
    if (p.lse && (p.fill & MC_FILL_LSE)) fill_lse(out, p.lse, p.H, p.T, w, warps);
  } else if (ROLE == kOutput) {
    // ------------------------------------------------------------ output
    // Warp w: rows 32 q .. 32 q + 31 of both tiles, O / row sum, while the other
    // warps are at the next item.
    const int q = warp & 3, row = q * 32 + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const long long st[3] = {p.os[0], p.os[1], 0};
    const bool wide = rows_wide(p.o, st);
    uint32_t no[2] = {0, 0};
    bool ok = true;
    for (uint32_t li = 0; ok; ++li) {
      Item x;
      if (!(ok = ring_get(ring, li, x, &abort_flag)) || x.head < 0) break;
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const Tile tl = tile_of(p, x, t);
        if (tl.nkv == 0) continue;
        const uint32_t par = no[t]++ & 1;
        if (!(ok = warp_wait(&l_full[t], par, &abort_flag) && warp_wait(&o_full[t], par, &abort_flag))) break;
        tc_fence_after();
        const float scale = inv[t * BM + row];
        const int i = tl.row0 + row;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + (x.b.start + i) * p.os[0] + tl.head * p.os[1];
#pragma unroll 1
        for (int col = 0; col < p.d_v; col += 32) store_rows(tmem + kO + t * BM + lanes + col, o + col, scale, i < x.b.len, wide, p.d_v - col);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_empty[t]);
      }
    }
    if (!ok && lane == 0) fail();
  } else if (ROLE == kSoftmax) {
    // ------------------------------------------------------------ softmax
    const int t = (warp - 8) >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t ts = tmem + t * BM + ((uint32_t)(q * 32) << 16), to = ts + kO;
    const float c2 = p.scale * kLog2e;
    const unsigned long long c22 = two(c2, c2);
    uint32_t ns = 0, no = 0;
    bool ok = true;
    unsigned long long z = 0;            // zeros, or NaN once a logit of the diagonal blocks is not finite
    bool bad = false;
    for (uint32_t li = 0;; ++li) {
      Item x;
      if (!(ok = ring_get(ring, li, x, &abort_flag)) || x.head < 0) break;
      const Tile tl = tile_of(p, x, t);
      if (tl.nkv == 0) continue;
      float m = -INFINITY, top = -INFINITY;
      unsigned long long l2 = 0;         // two halves of the row sum
      for (int j = 0; j < tl.nkv; ++j) {
        if (!(ok = warp_wait(&s_full[t], ns++ & 1, &abort_flag))) break;
        tc_fence_after();
        uint32_t r[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32_async(ts + 32 * c, r[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(r[c]);
        // the diagonal block: keys up to the row's own.  Of its four groups of 32 columns a
        // warp (rows 32 q ..) sees those before q whole, of q those up to the row, and none
        // behind.  Every token's own logit is here, so a NaN/Inf in its q or k shows here
        const bool diagonal = j == tl.nkv - 1;
        const int groups = diagonal ? q + 1 : 4;
        if (diagonal) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (g == q) {
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                z = fma2(two(c <= lane ? __uint_as_float(r[g][c]) : 0.f, 0.f), 0, z);
                if (c > lane) r[g][c] = 0xff800000u;
              }
            } else if (g < q) {
#pragma unroll
              for (int c = 0; c < 32; c += 2) z = fma2(two(__uint_as_float(r[g][c]), __uint_as_float(r[g][c + 1])), 0, z);
            }
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g >= groups) break;
#pragma unroll
          for (int c = 0; c < 32; c += 2) mx[c / 2 % 4] = max3f(mx[c / 2 % 4], __uint_as_float(r[g][c]), __uint_as_float(r[g][c + 1]));
        }
        const float mj = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        top = fmaxf(top, mj);
        const bool grow = mj * c2 > m + kLazy;      // always in the first block
        if (__any_sync(0xffffffffu, grow)) {
          const float m1 = grow ? mj * c2 : m, a = ex2_approx(m - m1);
          l2 = mul2(l2, two(a, a));
          m = m1;
          if (j > 0) {                   // S is complete, so the product before it, which wrote O, is too
#pragma unroll 1
            for (int col = 0; col < 64 * NCV; col += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16_async(to + col, o);
              tmem_ld_wait();
              reg_fence16(o);
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * a);
              tmem_st_32x32b_x8(to + col, o);
              tmem_st_32x32b_x8(to + col + 8, o + 8);
            }
          }
        }
        const unsigned long long nm = two(-m, -m);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t w[16];
          if (g < groups) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float p0, p1;
              untwo(fma2(two(__uint_as_float(r[g][2 * k]), __uint_as_float(r[g][2 * k + 1])), c22, nm), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              l2 = add2(l2, two(p0, p1));
              w[k] = pack_bf16(p0, p1);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = 0u;
          }
          tmem_st_32x32b_x8(ts + 16 * g, w);
          tmem_st_32x32b_x8(ts + 16 * g + 8, w + 8);
          if (g == 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[t]);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      float l, l1;
      untwo(l2, l, l1);
      l += l1;
      const int i = tl.row0 + row;
      const bool there = i < x.b.len;
      bad |= there && !(l <= 3.4e38f);   // NaN or +Inf among the logits
      // the output warps have read the previous item's row sums
      if (!(ok = warp_wait(&o_empty[t], (no++ & 1) ^ 1, &abort_flag))) break;
      inv[t * BM + row] = 1.f / l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&l_full[t]);
      if (p.lse && there) p.lse[(long long)tl.head * p.T + x.b.start + i] = (m + log2f(l)) * kLn2;
      float wm = there ? top : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
      if (lane == 0 && wm > -INFINITY) {
        // as float max orders them: non-negative values as signed, negative ones as unsigned integers
        const float v = wm * p.scale;
        if (__float_as_int(v) >= 0) atomicMax(reinterpret_cast<int*>(p.smax) + tl.head, __float_as_int(v));
        else atomicMin(reinterpret_cast<unsigned int*>(p.smax) + tl.head, __float_as_uint(v));
      }
    }
    if (!ok && lane == 0) fail();
    float z0, z1;
    untwo(z, z0, z1);
    if (__any_sync(0xffffffffu, bad || z0 != 0.f || z1 != 0.f) && lane == 0) set_status(p.status, MC_STATUS_NONFINITE_LOGIT);   // NaN differs from 0
  }
  tc_fence_before();
  block_sync();
  tc_fence_after();
}

template <int NCH, int NCV>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(const __grid_constant__ PackedFwdParams p, const __grid_constant__ Maps mp) {
  static_assert(smem_bytes(NCH, NCV) + 64 <= 227 * 1024, "shared memory");
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
  const uint32_t tmem = tmem_slot;
  await_previous();
  if (warp < 4) {
    regs_release<kRegsIssue>();
    forward<NCH, NCV, kIssue>(p, mp, smem, tmem, abort_flag, warp, lane);
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  } else if (warp < 8) {
    regs_release<kRegsOutput>();
    forward<NCH, NCV, kOutput>(p, mp, smem, tmem, abort_flag, warp, lane);
  } else {
    regs_acquire<kRegsSoftmax>();
    forward<NCH, NCV, kSoftmax>(p, mp, smem, tmem, abort_flag, warp, lane);
  }
}

template <int NCH, int NCV>
cudaError_t launch_fwd(const PackedFwdParams& p, const Maps& mp, int grid, cudaStream_t s) {
  constexpr size_t smem = smem_bytes(NCH, NCV);
  const cudaError_t e = cudaFuncSetAttribute(fwd_kernel<NCH, NCV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_behind(fwd_kernel<NCH, NCV>, (unsigned)grid, kThreads, smem, s, p, mp);
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

}  // namespace pf
}  // namespace

namespace packed {
bool encode_rows(CUtensorMap* m, const void* base, int width, int heads, long long T, const long long* st, int rows) {
  pf::EncodeTiledFn enc = pf::get_encode();
  if (!enc) return false;
  cuuint64_t dims[5] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)kFar, (cuuint64_t)T + 1, (cuuint64_t)kFar + 1};
  cuuint64_t by[4] = {(cuuint64_t)st[1] * 2, (cuuint64_t)st[0] * 2, (cuuint64_t)st[0] * 2, ((1ull << 34) - (cuuint64_t)st[0]) * 2};
  cuuint32_t box[5] = {64, 1, (cuuint32_t)rows, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return encode_bound([&] {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, by, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}
}  // namespace packed

cudaError_t launch_packed_plan(const PackedPlan& p, cudaStream_t s) {
  PackedPlan q = p;
  const size_t bytes = (2 * (size_t)p.nseq + p.capacity + 2) * 4;
  q.local = bytes <= pf::kPlanLocal;
  return launch_behind(pf::plan_kernel, 1u, (unsigned)pf::kPlanThreads, q.local ? bytes : 0, s, q);
}

cudaError_t launch_packed_fwd(const PackedFwdParams& p, int blocks, cudaStream_t s, char* err, size_t errlen) {
  using namespace pf;
  Maps mp;
  memset(&mp, 0, sizeof mp);
  const int Hkv = p.H / p.group;
  if (!packed::encode_rows(&mp.q, p.q, p.d, p.H, p.T, p.qs, BM) || !packed::encode_rows(&mp.k, p.k, p.d, Hkv, p.T, p.ks, BM) ||
      !packed::encode_rows(&mp.v, p.v, p.d_v, Hkv, p.T, p.vs, BM)) {
    snprintf(err, errlen, "tensor map encoding failed");
    return cudaErrorInvalidValue;
  }
  const long long items = (long long)blocks * p.order.heads;
  const int grid = (int)(items < sm_count() ? items : sm_count());
  const int nch = (p.d + 63) / 64, ncv = (p.d_v + 63) / 64;
  using Launch = cudaError_t (*)(const PackedFwdParams&, const Maps&, int, cudaStream_t);
  static const Launch by_chunks[2][2] = {{launch_fwd<1, 1>, launch_fwd<1, 2>}, {launch_fwd<2, 1>, launch_fwd<2, 2>}};
  return by_chunks[nch - 1][ncv - 1](p, mp, grid, s);
}

}  // namespace mc
