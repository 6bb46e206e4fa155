// Pieces shared by the varlen prefill kernels: the tcgen05 and TMEM wrappers
// in inline PTX, packed fp32 arithmetic, and the longest-first work order.
#pragma once

#include <cuda.h>

#include "pa_common.cuh"

namespace pa {

constexpr int kPfRows = 128;  // M: rows of a query tile
constexpr int kPfKeys = 64;   // keys per KV tile (N of the score MMA)

// mbar_wait where the phase is most likely over, or soon to be: the first try,
// which the hardware suspends for a while, stands alone in the instruction
// stream and the rest out of its way.
__device__ __forceinline__ bool mbar_wait_soon(uint32_t bar, uint32_t parity, volatile int *abort,
                                               int32_t *err) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  return mbar_wait(bar, parity, abort, err);
}

// ---- tcgen05 helpers ----------------------------------------------------------

// Shared-memory matrix descriptor (K- or MN-major, 128-byte swizzle):
// start address, leading / stride byte offsets (>> 4), version 1, layout 2.
__device__ __forceinline__ uint64_t umma_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for tcgen05
  d |= (uint64_t)2 << 61;  // SWIZZLE_128B
  return d;
}

// Instruction descriptor, kind::f16: bf16 A and B, fp32 D, M = 128, N = n,
// A K-major, B K-major (b_mn = 0) or MN-major (b_mn = 1).
__host__ __device__ constexpr uint32_t umma_idesc(int b_mn, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kPfRows >> 4) << 24);
}

// The MMA, commit and TMA helpers below are executed by a whole converged
// warp whose role branch the compiler can see is warp-uniform: every lane
// computes the same operands (kept in uniform registers) and one lane, picked
// by elect.sync, issues.  Issued from a lone lane in a divergent branch, each
// MMA cost about three times its tensor-pipe time.
//
// D (+)= A B with A (M x 16, K-major, two bf16 per 32-bit column) read from
// tensor memory at column address a_tmem and B described by b.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D (+)= A B with both operands described in shared memory.
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 64 consecutive fp32 columns of this thread's TMEM lane (two loads, one wait).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[2][32]) {
  uint32_t r[64];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[32 * h + 0]), "=r"(r[32 * h + 1]), "=r"(r[32 * h + 2]), "=r"(r[32 * h + 3]),
          "=r"(r[32 * h + 4]), "=r"(r[32 * h + 5]), "=r"(r[32 * h + 6]), "=r"(r[32 * h + 7]),
          "=r"(r[32 * h + 8]), "=r"(r[32 * h + 9]), "=r"(r[32 * h + 10]), "=r"(r[32 * h + 11]),
          "=r"(r[32 * h + 12]), "=r"(r[32 * h + 13]), "=r"(r[32 * h + 14]),
          "=r"(r[32 * h + 15]), "=r"(r[32 * h + 16]), "=r"(r[32 * h + 17]),
          "=r"(r[32 * h + 18]), "=r"(r[32 * h + 19]), "=r"(r[32 * h + 20]),
          "=r"(r[32 * h + 21]), "=r"(r[32 * h + 22]), "=r"(r[32 * h + 23]),
          "=r"(r[32 * h + 24]), "=r"(r[32 * h + 25]), "=r"(r[32 * h + 26]),
          "=r"(r[32 * h + 27]), "=r"(r[32 * h + 28]), "=r"(r[32 * h + 29]),
          "=r"(r[32 * h + 30]), "=r"(r[32 * h + 31])
        : "r"(taddr + 32 * h));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 32; ++i) v[h][i] = __uint_as_float(r[32 * h + i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
      "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
      "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
      "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
      "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
      "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 consecutive 32-bit columns of this thread's TMEM lane; completes at the
// next tmem_wait_st().
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Packed pairs of floats (lo half first) and the f32x2 arithmetic on them:
// each half is rounded as the scalar instruction would round it.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// max of three floats (exact; a NaN operand is ignored, as by fmaxf)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x by the special-function unit (ex2.approx, relative error ~2^-22).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of (row, 16-byte chunk) inside a [128 rows][128 B] swizzled half.
__device__ __forceinline__ uint32_t sw128(int row, int chunk) {
  return row * 128 + ((chunk ^ (row & 7)) << 4);
}

// ---- work order -------------------------------------------------------------
// The work items are (sequence s, query tile mt, kv head g) with a query
// tile of PT positions; an item costs one step per 64-key tile it attends,
// nkv = (prefix + last position of the tile) / 64 + 1, which grows with mt.
// CTAs start in block-index order, so the CTA of linear index r takes the
// item of rank r in the order "most steps first" (ties: by s, then mt, then
// g): long items start first and short ones fill the end of the grid.  Every
// CTA finds its item from a histogram of the step counts (one thread per
// sequence, counts clamped to kLptBins - 1, which only merges ties) and two
// block scans; a kernel of NT threads uses it only while num_seqs <= NT, so
// that this prologue stays one round of loads.  Returns false when the CTA has no item.  Sequences
// with rows beyond the grid's tiles or with context_lens < q_len are
// reported (PA_DEVERR_SHAPE); the latter have no items.
constexpr int kLptBins = 1024;
constexpr int kWorkOrderBytes = (kLptBins + 32 + 5) * 4;  // scratch of pick_work_item
__device__ __forceinline__ int lpt_bin(int prefix, int q_len, int mt, int PT) {
  const int last = mt * PT + min(PT, q_len - mt * PT) - 1;  // last position of the tile
  return min((prefix + last) / kPfKeys + 1, kLptBins - 1);
}
// exclusive block scan of one int per thread (NT threads)
template <int NT>
__device__ __forceinline__ int block_excl_scan(int v, int *wsum, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = lane < NT / 32 ? wsum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    if (lane < NT / 32) wsum[lane] = t;  // inclusive warp prefix
  }
  __syncthreads();
  total = wsum[NT / 32 - 1];
  const int before = warp > 0 ? wsum[warp - 1] : 0;
  __syncthreads();  // wsum is reused by the next scan
  return before + x - v;
}
template <int PT, int NT, bool kPlain = false, typename Params>
__device__ bool pick_work_item(const Params &p, int gx, int *sc, int &s_out, int &mt_out,
                               int &g_out) {
  int *hist = sc;                     // [kLptBins] items per step count
  int *wsum = sc + kLptBins;          // [NT / 32] block-scan scratch
  int *res = sc + kLptBins + 32;      // picked bin, items before it, s, mt, g
  const int tid = threadIdx.x;
  const int r = (int)(blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z));
  for (int i = tid; i < kLptBins; i += NT) hist[i] = 0;
  if (tid == 0) res[0] = -1;
  __syncthreads();
  const int ns = p.num_seqs, hkv = p.hkv;
  const int spt = (ns + NT - 1) / NT;
  const int s0 = min(ns, tid * spt), s1 = min(ns, s0 + spt);
  // pass 1: the histogram (runs of equal counts added at once)
  for (int s = s0; s < s1; ++s) {
    const int q_len = ld_index<kPlain>(p.cu_seqlens + s + 1) - ld_index<kPlain>(p.cu_seqlens + s);
    if (q_len <= 0) continue;
    const int prefix = ld_index<kPlain>(p.context_lens + s) - q_len;
    if (prefix < 0) {
      report(p.err, PA_DEVERR_SHAPE);
      continue;
    }
    if (q_len > gx * PT) report(p.err, PA_DEVERR_SHAPE);  // rows no CTA covers
    const int T = min((q_len + PT - 1) / PT, gx);
    int run_bin = lpt_bin(prefix, q_len, 0, PT), run = 0;
    for (int mt = 0; mt < T; ++mt) {
      const int b = lpt_bin(prefix, q_len, mt, PT);
      if (b != run_bin) {
        atomicAdd(hist + run_bin, run * hkv);
        run_bin = b;
        run = 0;
      }
      ++run;
    }
    if (T > 0) atomicAdd(hist + run_bin, run * hkv);
  }
  __syncthreads();
  // pass 2 (warp 0): the bin of rank r, counting bins from the top
  if (tid < 32) {
    constexpr int kPer = kLptBins / 32;
    int sum = 0;
#pragma unroll 4
    for (int k = 0; k < kPer; ++k) sum += hist[kLptBins - 1 - tid * kPer - k];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += y;
    }
    const int excl = incl - sum;
    if (r >= excl && r < incl) {
      int acc = excl;
      for (int k = 0; k < kPer; ++k) {
        const int b = kLptBins - 1 - tid * kPer - k;
        if (r < acc + hist[b]) {
          res[0] = b;
          res[1] = acc;
          break;
        }
        acc += hist[b];
      }
    }
  }
  __syncthreads();
  const int vb = res[0];
  if (vb < 0) return false;  // rank past the last item
  const int j = r - res[1];
  // pass 3: the j-th item of bin vb in (s, mt, g) order
  int cnt = 0;
  for (int s = s0; s < s1; ++s) {
    const int q_len = ld_index<kPlain>(p.cu_seqlens + s + 1) - ld_index<kPlain>(p.cu_seqlens + s);
    const int prefix = ld_index<kPlain>(p.context_lens + s) - q_len;
    if (q_len <= 0 || prefix < 0) continue;
    const int T = min((q_len + PT - 1) / PT, gx);
    for (int mt = 0; mt < T; ++mt) cnt += lpt_bin(prefix, q_len, mt, PT) == vb ? hkv : 0;
  }
  int total;
  const int before = block_excl_scan<NT>(cnt, wsum, total);
  if (j >= before && j < before + cnt) {
    int k = j - before;
    for (int s = s0; s < s1 && k >= 0; ++s) {
      const int q_len = ld_index<kPlain>(p.cu_seqlens + s + 1) - ld_index<kPlain>(p.cu_seqlens + s);
      const int prefix = ld_index<kPlain>(p.context_lens + s) - q_len;
      if (q_len <= 0 || prefix < 0) continue;
      const int T = min((q_len + PT - 1) / PT, gx);
      for (int mt = 0; mt < T; ++mt) {
        if (lpt_bin(prefix, q_len, mt, PT) != vb) continue;
        if (k < hkv) {
          res[2] = s;
          res[3] = mt;
          res[4] = k;
          k = -1;
          break;
        }
        k -= hkv;
      }
    }
  }
  __syncthreads();
  s_out = res[2];
  mt_out = res[3];
  g_out = res[4];
  // the scratch becomes a TMA destination: order these generic writes first
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return true;
}

}  // namespace pa
