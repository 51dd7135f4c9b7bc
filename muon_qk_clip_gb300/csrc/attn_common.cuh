// Device helpers that the attention kernels share: products with an operand in
// tensor memory, register shares, elected lanes, warp-wide waits and the way of an
// accumulator from tensor memory to bf16 rows.
#pragma once

#include "common.cuh"

namespace mc {
namespace attn {

// D[tmem] (+)= A[tmem] * B[smem]^T: A is M rows (lanes) of bf16 pairs, K-major.
__device__ inline void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <int N>
__device__ inline void regs_release() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ inline void regs_acquire() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// True in one lane of the (whole) warp.  The MMA issuer runs as a whole warp
// with the products under this predicate, so that descriptors stay in uniform
// registers.
__device__ inline bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// 32 lanes x 8 columns of 32-bit values into TMEM
__device__ inline void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ inline uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h2);
}

// All 32 lanes wait; true only if every lane saw the phase complete.
__device__ inline bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = mbar_wait(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, ok);
}
// 32 columns of 32 lanes, waited for.
__device__ inline void load_32(uint32_t taddr, uint32_t (&r)[2][16]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x16_async(taddr + c * 16, r[c]);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 2; ++c) reg_fence16(r[c]);
}
// One 32-byte sector (aligned)
__device__ inline void store_32b(void* to, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 32 columns of an accumulator, from tensor memory at `taddr` (a row per lane),
// times `scale`, as bf16, to this lane's row of an output at `dst`.  The row
// exists if `row`, and `n` of its columns.  Rows on 32-byte boundaries (`wide`) are
// stored a whole sector per lane and instruction.  True if a value of the row is
// not finite.
//
// The next item's products wait for the accumulators, so they leave tensor memory
// by the shortest way.  (Turned through shared memory, so that neighbouring lanes
// write neighbouring addresses, 32 columns took 900 clocks, most of them waiting
// for shared memory behind the tensor core's operand reads.)  The epilogue calls
// this in loops that stay rolled: its code runs once per work item between tiles
// of other code, and unrolled it spent most of its time fetching instructions.
__device__ inline bool store_rows(uint32_t taddr, __nv_bfloat16* dst, float scale, bool row, bool wide, int n) {
  uint32_t r[2][16], w[16];
  load_32(taddr, r);
  const unsigned long long s2 = two(scale, scale);
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 z = zero;               // zeros, or NaN once a value is not finite
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    float v0, v1;
    untwo(mul2(two(__uint_as_float(r[x / 8][2 * (x % 8)]), __uint_as_float(r[x / 8][2 * (x % 8) + 1])), s2), v0, v1);
    const __nv_bfloat162 v = __floats2bfloat162_rn(v0, v1);
    z = __hfma2(v, zero, z);
    w[x] = *reinterpret_cast<const uint32_t*>(&v);
  }
  if (row) {
    if (wide && n >= 32) {
#pragma unroll
      for (int u = 0; u < 2; ++u) store_32b(dst + 16 * u, w + 8 * u);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (8 * u + 8 <= n) {
          *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        } else {
#pragma unroll
          for (int y = 0; y < 7; ++y)
            if (8 * u + y < n) dst[8 * u + y] = __ushort_as_bfloat16((unsigned short)(w[4 * u + y / 2] >> (16 * (y % 2))));
        }
      }
    }
  }
  __syncwarp();
  return row && (__low2float(z) != 0.f || __high2float(z) != 0.f);   // NaN differs from 0
}
// Whether every row of an output begins on a 32-byte boundary (its blocks of 32
// columns then do too).
__device__ inline bool rows_wide(const void* base, const long long* st) {
  return ((reinterpret_cast<uintptr_t>(base) >> 1 | (uintptr_t)st[0] | (uintptr_t)st[1] | (uintptr_t)st[2]) & 15) == 0;
}

}  // namespace attn
}  // namespace mc
