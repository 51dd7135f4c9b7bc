// What the packed attention's forward and backward share: the plan of a call's
// row blocks, ragged tensor maps and the hand-out of work items.
#pragma once

#include "attn_common.cuh"
#include "common.cuh"

namespace mc {
namespace packed {

// One block of query (or key) rows of one sequence.
struct Block {
  int start, len;      // the sequence's first token and length
  int index;           // of the block within it
  int pad;             // the sequence's first place among padded rows (backward)
};

// A work item on its way through shared memory from the producer to the other
// warps of the block: block and head (head < 0: no more items).  As in the dense
// kernels, the producer takes the next item before it loads the current one's
// last tile.
constexpr int kRing = 4;
struct Item {
  Block b;
  int head;
};
constexpr int kSlot = 8;                 // ints per slot
struct Ring {
  volatile int* slot;                    // [kRing][kSlot]
  uint64_t* full;                        // [kRing] 1 arrival
  uint64_t* empty;                       // [kRing] an arrival from each of the 13 other warps
};
__device__ inline bool ring_put(const Ring& r, uint32_t n, const Item& x, volatile int* abort_flag) {
  const int s = n % kRing;
  if (!mbar_wait(&r.empty[s], ((n / kRing) & 1) ^ 1, abort_flag)) return false;
  volatile int* to = r.slot + s * kSlot;
  to[0] = x.b.start; to[1] = x.b.len; to[2] = x.b.index; to[3] = x.b.pad; to[4] = x.head;
  mbar_arrive(&r.full[s]);
  return true;
}
// The n-th item for a whole warp; false on a wait that gave up.
__device__ inline bool ring_get(const Ring& r, uint32_t n, Item& x, volatile int* abort_flag) {
  const int s = n % kRing;
  if (!attn::warp_wait(&r.full[s], (n / kRing) & 1, abort_flag)) return false;
  const volatile int* at = r.slot + s * kSlot;
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };    // the same in every lane, and uniform to the compiler
  x.b.start = uniform(at[0]); x.b.len = uniform(at[1]); x.b.index = uniform(at[2]); x.b.pad = uniform(at[3]); x.head = uniform(at[4]);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[s]);
  return true;
}

// Work order.  The plan lists the blocks heaviest first; an item is a block and a
// head (or pair of heads), the heads of a group next to each other: those whose
// keys and values L2 can hold together.  A block that does not lie within the T
// tokens (the workspace was written by others meanwhile) ends the work.
__device__ inline Item item_at(const Block* blocks, int count, const Order& o, int T, int rows, int x) {
  Item it;
  it.b = Block{0, 0, 0, 0};
  it.head = -1;
  if (count <= 0 || x >= count * o.heads) return it;
  const int per = count * o.group;
  const int g = x / per, rem = x - g * per, n = min(o.group, o.heads - g * o.group), e = rem / n;
  const int4 b = *reinterpret_cast<const int4*>(blocks + e);
  if (b.x < 0 || b.y < 1 || b.x > T - b.y || b.z < 0 || b.z > (b.y - 1) / rows) return it;
  it.b = Block{b.x, b.y, b.z, b.w};
  it.head = g * o.group + (rem - e * n);
  return it;
}

// Rows [first, first + R) of a sequence as a tile of R rows, those past its end as
// zeros.  The tokens of all sequences lie behind one another, so the bound that the
// copy checks is not the end of an axis of tokens.  The map has the token stride on
// an axis of kFar rows and again on one of places: row coordinate kFar - n and place
// first + n (n: rows that exist) address row `first`, kFar rows too far, and the
// copy runs over the end of the row axis after n rows.  A last axis takes the kFar
// rows back: its stride is 2^34 elements less the token stride, and at coordinate
// kFar = 2^30 that is 2^64 elements less kFar token strides.  (A map whose base lies R
// rows before the tensor needs no such axis, but a tensor near the start of its
// allocation faulted with one, although no coordinate reached the rows before it.)
constexpr int kFar = 1 << 30;
template <int R>
__device__ inline void load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int chunk, int head, const Block& b, int first) {
  const int n = min(R, b.len - first);
  tma_load_5d(dst, map, bar, 64 * chunk, head, kFar - n, b.start + first + n, kFar);
}

// Tokens that belong to no sequence: sequences lie one behind the other, so these are the
// ones in front of the first and behind the last.  Their rows are set by warps that have nothing else to
// do, beside the items' work.
struct Outside {
  int first, last, n;
};
__device__ inline Outside outside_of(const int* count, int T) {
  Outside x;
  x.first = min(max(count[1], 0), T);
  x.last = min(max(count[2], x.first), T);
  x.n = x.first + T - x.last;
  return x;
}
// Zeros in an output [T, heads, width]; warp `w` of `warps`, half a warp per row.
__device__ inline void fill_rows(const Outside& x, void* base, const long long* st, int heads, int width, int w, int warps) {
  const int lane = threadIdx.x & 31, c = 8 * (lane & 15);
  for (int i = w; i < x.n; i += warps) {
    const int t = i < x.first ? i : x.last + (i - x.first);
    for (int h = lane >> 4; h < heads; h += 2) {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(base) + t * st[0] + h * st[1];
      if (c + 8 <= width) {
        *reinterpret_cast<uint4*>(row + c) = make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (int y = c; y < width; ++y) row[y] = __ushort_as_bfloat16(0);
      }
    }
  }
}
// -inf in lse [H, T].
__device__ inline void fill_lse(const Outside& x, float* lse, int H, int T, int w, int warps) {
  if (x.n == 0) return;
  const long long all = (long long)H * x.n;
  for (long long e = (long long)w * 32 + (threadIdx.x & 31); e < all; e += (long long)warps * 32) {
    const int h = (int)(e / x.n), i = (int)(e - (long long)h * x.n);
    lse[(long long)h * T + (i < x.first ? i : x.last + (i - x.first))] = -INFINITY;
  }
}

// Host: such a map of [T, heads, width] with strides (token, head), R rows.
bool encode_rows(CUtensorMap* m, const void* base, int width, int heads, long long T, const long long* st, int rows);

}  // namespace packed
}  // namespace mc
