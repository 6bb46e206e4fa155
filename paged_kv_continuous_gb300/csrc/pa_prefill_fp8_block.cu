// pa_prefill_fp8_block: causal varlen attention of cu_seqlens-packed query
// chunks over a block-scaled FP8 cache (pa_fp8_block.cuh), on tcgen05.
//
// One CTA computes a 128-row tile of one (sequence, kv head), rows being the
// (query position, query head) pairs of 128 / G positions, over 64-key tiles:
//   S   = (Q_hi + Q_lo) C_k^T   e4m3 x e4m3 -> fp32 (C: codes)
//   t   = c 2^(eq + ek) S + ev  base-2 score plus the exponent of V's scale
//   P'  = 2^(t - m)             m the row's running reference of t
//   O  += P' C_v                f16 x f16 -> fp32 in TMEM
//   l  += 2^-ev P'              per 16-key page;        out = O / l.
// Neither scale is applied to an element: K's goes into the page's factor of
// the exponent, V's into its offset, so P' <= 256 carries weight times V
// scale relative to the largest such product, and one f16 term of it (11
// bits) suffices for a 4-bit significand.
//
// K codes feed the score MMA as they are: a query row times 2^-eq, its
// largest magnitude in (224, 448], is the sum of two E4M3 terms.  A bf16 has 8
// significant bits; the rounded first term leaves a remainder of at most 4
// bits, which the second holds exactly wherever the element is at least 2^-9
// of the row's largest (the last inexact one is 0.249 where the largest is 226;
// below, the error is under 2^-17 of the largest).  Two passes at the FP8 rate
// cost what one f16 pass would, and K needs no conversion: its pages arrive by
// TMA in the layout the MMA reads.
//
// V codes are widened to f16 by one warp, from a staging buffer that bulk
// copies fill (a page of a head is 2 KB contiguous).  V pages are dim-major,
// [128 dims][16 tokens]: K-major rows (a dim, 64 keys = 128 bytes) of the PV
// MMA with no transpose, written in the 128-byte swizzle.
//
// Warps: 0 requests pages (K boxes, V staging) and scales, 1 issues the score
// MMAs, 3 the PV MMAs, 2 widens V, 4 .. 7 run the softmax, a row per thread.
// Two CTAs share an SM: one's softmax runs while the other's MMAs use the
// tensor pipe.
//
// What bounds it (two chunks of 2 k queries behind 15 k keys, Hq 32, Hkv 8:
// 823 us, 1.18 PFLOP/s causal): a 64-key step of both CTAs of an SM takes about
// 1630 cycles, of which the tensor pipe is busy about 1280 (the score MMAs at N
// = 64 read their A and B tiles from shared memory at 48 cycles each, against
// 32 of arithmetic), and the latency of the single warps' instruction streams
// sets the rest; the last of four waves of CTAs is a sixth full.  Tried: two
// warps widening K and V from plain loads into f16 tiles, 2068 us (the loads'
// latency); scale bytes loaded tile by tile, 1366 us (the same, in warp 0); one
// election per TMA or MMA and page loops, 1147 us; one issuer for both MMAs and
// two widening warps, 1040 us; V requested by the widening warp, 1090 us, or by
// the PV warp, 931 us; P' in a rolled loop that reads the scores twice, 1055 us;
// the widening's loads a page ahead, 927 us.
//
// A NaN code of a value may only reach the rows that see its key, but in the MMA
// 0 * NaN is NaN.  So the widening warp looks through the few tiles that the
// causal limit cuts (two of 270 in a long chunk), turns NaN codes past the query
// tile's first position into zeros and keeps the first such key of each dim; the
// rows that see it write NaN there at the end.  The rest of that is out of line:
// inlined, it moved registers of the tile loops, 2 % (and 14 % for a search by the
// softmax threads before they start).  As it is, the long case takes 824 us
// against 812 without, the mixed one 54.5 against 54.9, timed in turn.  A query row
// with a NaN or an infinity gives NaN.
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "pa_fp8_block.cuh"
#include "pa_prefill_common.cuh"

namespace pa {
namespace {

constexpr int kQpThreads = 256;
constexpr int kQpSoft = 128;                    // softmax threads
constexpr int kQpPages = kPfKeys / kBlockSize;  // pages per KV tile
constexpr int kQpCodes = kPfKeys * kHeadDim;    // one K or V tile of codes: 8 KB
constexpr int kQpPage = kBlockSize * kHeadDim;  // one page of one head: 2 KB
constexpr int kQpTile = 2 * kQpCodes;           // one V tile, f16: 128 dims x 64 keys
constexpr int kQpQ = kPfRows * kHeadDim;        // one E4M3 term of Q: 128 rows x 128 bytes
// two K stages (codes), three stages of V codes, two of widened V: 104 KB with
// Q, under half an SM's
constexpr int kQpKStages = 2, kQpCStages = 3, kQpVStages = 2;
constexpr int kQpOffQ = 0;
constexpr int kQpOffK = kQpOffQ + 2 * kQpQ;
constexpr int kQpOffC = kQpOffK + kQpKStages * kQpCodes;  // V codes
constexpr int kQpOffV = kQpOffC + kQpCStages * kQpCodes;
constexpr int kQpOffBar = kQpOffV + kQpVStages * kQpTile;
// 8-byte slots: K full / empty per stage, V codes full / empty, widened V full
// / empty, Q ready, two score, two P and two PV barriers, eight scale
// barriers, TMEM address, abort flag; then the page scales of eight tiles (K's
// four bytes, V's four).  From kQpOffNan on the first NaN key of each dim, and in
// the word before whether there is one.
constexpr int kSlKFull = 0, kSlKEmpty = kSlKFull + kQpKStages;
constexpr int kSlCFull = kSlKEmpty + kQpKStages, kSlCEmpty = kSlCFull + kQpCStages;
constexpr int kSlVFull = kSlCEmpty + kQpCStages, kSlVEmpty = kSlVFull + 2;
constexpr int kSlQ = kSlVEmpty + 2, kSlS = kSlQ + 1, kSlP = kSlS + 2, kSlO = kSlP + 2;
constexpr int kSlScale = kSlO + 2, kSlTmem = kSlScale + 8, kSlAbort = kSlTmem + 1;
constexpr int kSlScales = kSlAbort + 1;
constexpr int kQpOffNan = kQpOffBar + 512;
constexpr int kQpBarBytes = 512 + 4 * kHeadDim;
static_assert((kSlScales + 8) * 8 + 4 <= 512, "barrier slots do not fit");
constexpr int kQpSmem = 1024 + kQpOffBar + kQpBarBytes;
// TMEM (256 columns, two CTAs per SM): scores of tile j in buffer j % 2 at 0
// and 64, P' over the scores it came from (32 columns, two keys each), O at 128
constexpr int kQpTmemCols = 256, kQpTmemS = 64, kQpTmemO = 128;

struct PrefillQParams {
  void *out;
  int out_f32;
  const uint16_t *q;
  const int32_t *cu_seqlens;
  int num_seqs;
  int total_tokens;
  int sms;
  const uint8_t *v_cache;
  const uint8_t *k_scale, *v_scale;
  long long num_blocks;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int hq, hkv;
  float qk_scale_log2;    // > 0: a scale <= 0 is folded into q as staged
  uint32_t q_and, q_xor;  // staged q pairs = (q & q_and) ^ q_xor
  int32_t *err;
  int max_context;  // keys that a table row has entries for
};

// Instruction descriptor, fp32 D, M = 128, N = n, both operands K-major and of
// format 0: f16 under kind::f16, e4m3 under kind::f8f6f4.
__host__ __device__ constexpr uint32_t idesc_format0(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kPfRows >> 4) << 24);
}

// The helpers below are executed by a whole converged warp; each issues a run
// of asynchronous instructions from one elected lane under a single election
// (an election per instruction made up most of the issuing warp's time).
//
// S = (Q_hi + Q_lo) K^T: two terms of A (kQpQ bytes apart) and one B, E4M3,
// four k-steps of 32 dims (32 bytes of each 128-byte row) each; then commits
// to two barriers.  `a` and `b` are descriptors of the first k-step.
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint64_t a, uint64_t b,
                                             uint32_t idesc, uint32_t bar0, uint32_t bar1) {
  asm volatile(
      "{\n\t.reg .pred e, n, y;\n\t.reg .b64 a1, a2, a3, b1, b2, b3, c0, c1, c2, c3;\n\t"
      "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "add.u64 c0, %1, %6;\n\tadd.u64 c1, a1, %6;\n\tadd.u64 c2, a2, %6;\n\t"
      "add.u64 c3, a3, %6;\n\t"
      "setp.ne.b32 n, 0, 0;\n\tsetp.eq.b32 y, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, n;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c0, %2, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c1, b1, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c2, b2, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], c3, b3, %3, y;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(bar0), "r"(bar1), "n"(kQpQ >> 4)
      : "memory");
}

// O (+)= P' V: A in TMEM (8 columns per k-step of 16 keys), B of f16 rows of
// 64 keys, four k-steps; then commits to two barriers.
__device__ __forceinline__ void issue_values(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate, uint32_t bar0,
                                             uint32_t bar1) {
  asm volatile(
      "{\n\t.reg .pred e, n, y;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
      "setp.ne.b32 n, %4, 0;\n\tsetp.eq.b32 y, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, n;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, y;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, y;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t}" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(bar0), "r"(bar1)
      : "memory");
}

// Four K pages (boxes at token slots z) to dst, kQpPage bytes apart.
__device__ __forceinline__ void load_k_pages(uint32_t dst, const CUtensorMap *map, int g,
                                             const int (&z)[4], uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 d1, d2, d3;\n\t"
      "add.u32 d1, %0, 2048;\n\tadd.u32 d2, %0, 4096;\n\tadd.u32 d3, %0, 6144;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%7], 8192;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {0, %2, %3}], [%7];\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [d1], [%1, {0, %2, %4}], [%7];\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [d2], [%1, {0, %2, %5}], [%7];\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [d3], [%1, {0, %2, %6}], [%7];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(g), "r"(z[0]), "r"(z[1]), "r"(z[2]), "r"(z[3]),
      "r"(bar)
      : "memory");
}

// Four V pages (2 KB each) to dst, kQpPage bytes apart.
__device__ __forceinline__ void load_v_pages(uint32_t dst, const uint8_t *const (&v)[4],
                                             uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 d1, d2, d3;\n\t"
      "add.u32 d1, %0, 2048;\n\tadd.u32 d2, %0, 4096;\n\tadd.u32 d3, %0, 6144;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], 8192;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 2048, "
      "[%5];\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [d1], [%2], 2048, "
      "[%5];\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [d2], [%3], 2048, "
      "[%5];\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [d3], [%4], 2048, "
      "[%5];\n\t}" ::"r"(dst),
      "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]), "r"(bar)
      : "memory");
}
static_assert(kQpPage == 2048 && kQpCodes == 8192 && kQpPages == 4, "page loads");

__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t codes) {  // low two bytes
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)(codes & 0xFFFFu)));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 codes_to_float2(uint32_t codes) {  // low two bytes, exact
  float lo, hi;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(f16x2_of_codes(codes)));
  return make_float2(lo, hi);
}
// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = r[i];
}
// Scale byte of a query row with largest magnitude a: as scale_for, over a
// span wide enough for any row that matters (2^-100 .. 2^100).
__device__ __forceinline__ int query_scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  const int byte = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(byte, kScaleBias - 100), kScaleBias + 100);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// Warp 0: the K pages (TMA boxes), the V pages (bulk copies: a page of a head
// is contiguous) and the scales of tiles 0 .. nkv - 1 of (sequence, kv head
// g).  The latency of this warp's own instructions can set the pace of the
// whole tile loop, so a tile is one shape: four pages, always.  A page with no
// key is page 0 in its place (nothing of it is used), and so is a bad entry,
// which is reported (its rows are unspecified).  Table entries come eight
// tiles (32 pages, one per lane) at a time, eight tiles ahead, and their
// scales four tiles ahead.
__device__ __forceinline__ void request_tiles(const PrefillQParams &p, const CUtensorMap *map,
                                              const int32_t *row, int n, int nkv, int g,
                                              uint32_t base, uint32_t slot0,
                                              volatile int *abort_flag) {
  const int lane = threadIdx.x & 31;
  auto slot = [&](int i) { return slot0 + 8 * i; };
  auto entries = [&](int j8) -> int {
    const int lb = j8 * 32 + lane;
    if (lb * kBlockSize >= n) return 0;
    const int x = lb < p.bt_stride ? row[lb] : -1;
    const bool ok = x >= 0 && x < p.num_blocks;
    if (!ok) report(p.err, PA_DEVERR_BLOCK_INDEX);
    return ok ? x : 0;
  };
  auto scales_of = [&](int x) -> uint32_t {  // K's byte, V's << 8
    const long long at = (long long)x * p.hkv + g;
    return (uint32_t)p.k_scale[at] | ((uint32_t)p.v_scale[at] << 8);
  };
  const uint8_t *v_head = p.v_cache + (long long)g * kQpPage;
  const long long v_page = (long long)p.hkv * kQpPage;
  int next = entries(0), ph = 0;
  uint32_t next_sc = scales_of(next), sc = 0;
  int k_asked = 0, c_asked = 0;  // tiles whose K, V pages were requested
  int st = 0, round = 0;         // stage of tile j's K pages, and its use
  int cs = 0, cround = 0;        // the same of its V codes
  for (int j = 0; j < nkv; ++j) {
    if ((j & 7) == 0) {
      ph = next;
      sc = clamp_scales4(next_sc);
      next = j + 8 < nkv ? entries((j >> 3) + 1) : 0;
    } else if ((j & 7) == 4) {
      next_sc = scales_of(next);
    }
    int z[4];
    const uint8_t *v[4];
#pragma unroll
    for (int pg = 0; pg < kQpPages; ++pg) {
      const int x = __shfl_sync(0xffffffffu, ph, (j & 7) * kQpPages + pg);
      z[pg] = x * kBlockSize;
      v[pg] = v_head + x * v_page;
    }
    if (round > 0 && !__all_sync(0xffffffffu, mbar_wait_soon(slot(kSlKEmpty + st),
                                                             (round - 1) & 1, abort_flag, p.err)))
      break;
    load_k_pages(base + kQpOffK + st * kQpCodes, map, g, z, slot(kSlKFull + st));
    k_asked = j + 1;
    if (++st == kQpKStages) {
      st = 0;
      ++round;
    }
    // the scales of tile j: slot j % 8, last read by the softmax of tile
    // j - 8, which is over (the K stage is free: the score MMA of tile j - 2
    // waited for the PV of tile j - 4)
    if ((lane >> 2) == (j & 7)) {
      const uint32_t at = slot(kSlScales + (j & 7)) + (lane & 3);
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(sc & 0xFFu) : "memory");
      asm volatile("st.shared.u8 [%0], %1;" ::"r"(at + 4), "r"((sc >> 8) & 0xFFu) : "memory");
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(slot(kSlScale + (j & 7)));
    __syncwarp();
    if (cround > 0 &&
        !__all_sync(0xffffffffu, mbar_wait_soon(slot(kSlCEmpty + cs), (cround - 1) & 1,
                                                abort_flag, p.err)))
      break;
    load_v_pages(base + kQpOffC + cs * kQpCodes, v, slot(kSlCFull + cs));
    c_asked = j + 1;
    if (++cs == kQpCStages) {
      cs = 0;
      ++cround;
    }
  }
  if (lane == 0 && *abort_flag) {
    // copies in flight land before the CTA's shared memory is released
    volatile int never = 0;
    for (int i = max(k_asked - kQpKStages, 0); i < k_asked; ++i)
      mbar_wait(slot(kSlKFull + i % kQpKStages), (i / kQpKStages) & 1, &never, nullptr);
    for (int i = max(c_asked - kQpCStages, 0); i < c_asked; ++i)
      mbar_wait(slot(kSlCFull + i % kQpCStages), (i / kQpCStages) & 1, &never, nullptr);
  }
  __syncwarp();
}

// High bit of each byte that is a NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_codes4(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// A staged V tile (its first key is key0) holds NaN codes: those past `seen`, the
// last key of the query tile's first row, become zeros, word `dim` at nan0 keeps
// the first of them, and the word before tells that there is one.
__device__ __noinline__ void take_nan_codes(uint32_t codes, uint32_t nan0, int key0, int seen) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) sts32(nan0 - 4, 1u);
#pragma unroll 1
  for (int c = 0; c < 16; ++c) {  // page c / 4, dims 32 (c % 4) + lane
    const int first = key0 + (c >> 2) * kBlockSize, past = seen + 1 - first;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {  // tokens 4 i .. 4 i + 3
      const int b = min(max(past - 4 * i, 0), 4);
      const uint32_t at = codes + c * 512 + 16 * lane + 4 * i;
      const uint32_t x = lds32(at);
      const uint32_t m = b >= 4 ? 0u : nan_codes4(x) & (0xFFFFFFFFu << (8 * b));
      if (!m) continue;
      sts32(at, x & ~((m >> 7) * 0xFFu));
      const int key = first + 4 * i + ((__ffs((int)m) - 1) >> 3);
      const uint32_t d = nan0 + 4 * (32 * (c & 3) + lane);
      if (key < (int)lds32(d)) sts32(d, (uint32_t)key);
    }
  }
  __syncwarp();
}

// Warp 2: the V codes of each tile to f16.
__device__ __forceinline__ void widen_v_tiles(const PrefillQParams &p, int n, int nkv, int seen,
                                              uint32_t base, uint32_t slot0,
                                              volatile int *abort_flag) {
  const int lane = threadIdx.x & 31;
  auto slot = [&](int i) { return slot0 + 8 * i; };
  int cs = 0, cround = 0;  // stage of the codes of tile j, and its use
  for (int j = 0; j < nkv; ++j) {
    const int st = j & 1;
    bool ok = mbar_wait_soon(slot(kSlCFull + cs), cround & 1, abort_flag, p.err);
    if (ok && j >= 2)
      ok = mbar_wait_soon(slot(kSlVEmpty + st), ((j >> 1) - 1) & 1, abort_flag, p.err);
    if (!__all_sync(0xffffffffu, ok)) return;
    if ((j + 1) * kPfKeys - 1 > seen) {
      uint32_t any = 0;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint4 w = lds128(base + kQpOffC + cs * kQpCodes + 16 * lane + c * 512);
        any |= nan_codes4(w.x) | nan_codes4(w.y) | nan_codes4(w.z) | nan_codes4(w.w);
      }
      if (__any_sync(0xffffffffu, any != 0))
        take_nan_codes(base + kQpOffC + cs * kQpCodes, base + kQpOffNan, j * kPfKeys, seen);
    }
    const uint32_t from = base + kQpOffC + cs * kQpCodes + 16 * lane;
    const uint32_t to = base + kQpOffV + st * kQpTile + lane * 128;
    // chunk q of a page: dims 32 q .. + 31, one per lane, 16 tokens
#pragma unroll 1
    for (int pg = 0; pg < kQpPages; ++pg) {
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = lds128(from + pg * kQpPage + q * 512);
      // tokens past the last key weigh 0 and may hold anything: zero codes
      const int left = n - (j * kPfKeys + pg * kBlockSize);
      if (left < kBlockSize) {
        uint32_t mask[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int keep = min(max(left - 4 * q, 0), 4);
          mask[q] = keep >= 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          w[q].x &= mask[0];
          w[q].y &= mask[1];
          w[q].z &= mask[2];
          w[q].w &= mask[3];
        }
      }
      // dim row 32 q + lane: chunks 2 pg and 2 pg + 1, swizzled by the row
      const uint32_t c0 = ((2 * pg) ^ (lane & 7)) << 4, c1 = c0 ^ 16;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sts128(to + q * 32 * 128 + c0, f16x2_of_codes(w[q].x), f16x2_of_codes(w[q].x >> 16),
               f16x2_of_codes(w[q].y), f16x2_of_codes(w[q].y >> 16));
        sts128(to + q * 32 * 128 + c1, f16x2_of_codes(w[q].z), f16x2_of_codes(w[q].z >> 16),
               f16x2_of_codes(w[q].w), f16x2_of_codes(w[q].w >> 16));
      }
    }
    // the codes are read; the widened tile is visible to the tensor core
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(slot(kSlVFull + st));
      mbar_arrive(slot(kSlCEmpty + cs));
    }
    if (++cs == kQpCStages) {
      cs = 0;
      ++cround;
    }
  }
}

// The work order.  Work items are (sequence s, query tile mt of PT positions,
// kv head g), an item's length the number of 64-key tiles it attends, and the
// CTA of linear index r takes the item of rank r, longest first (ties by s, mt,
// g), so that long items do not start at the end of the grid.  Lengths grow
// with mt, so the tiles of a sequence that are at least v long are a closed
// form; every warp finds the length of rank r by bisection over such counts and
// the item by one scan, a sequence per lane (kSeqsPerLane of them at most), with
// no barrier.  (With a histogram over all items in shared memory, 8 to 16
// thousand cycles a CTA, and registers spilled: sixteen mixed chunks 56.3 us
// against 54.9, two long ones 852 against 818.)
constexpr int kSeqsPerLane = 8;
struct WorkItem {
  int s, mt, g;  // s < 0: none
};
template <int PT>
__device__ __forceinline__ WorkItem pick_item(const PrefillQParams &p, int gx, int r) {
  const int lane = threadIdx.x & 31;
  const int per = (p.num_seqs + 31) / 32;
  int prefix[kSeqsPerLane], q_len[kSeqsPerLane];
  int longest = 0;
#pragma unroll
  for (int k = 0; k < kSeqsPerLane; ++k) {
    prefix[k] = q_len[k] = 0;
    const int s = lane * per + k;
    if (k < per && s < p.num_seqs) {
      const int q = p.cu_seqlens[s + 1] - p.cu_seqlens[s];
      const int pre = max(p.context_lens[s], 0) - q;
      // (reported once, by the CTA of rank 0; q < 0: cu_seqlens that fall)
      if (r == 0 && threadIdx.x < 32 && (pre < 0 || (unsigned)q > (unsigned)(gx * PT)))
        report(p.err, PA_DEVERR_SHAPE);
      if (q > 0 && pre >= 0) {
        prefix[k] = pre;
        q_len[k] = q;
        longest = max(longest, (pre + min(q, gx * PT) - 1) / kPfKeys + 1);
      }
    }
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  // tiles of the lane's k-th sequence in the grid, and those shorter than v
  auto tiles = [&](int k) { return min((q_len[k] + PT - 1) / PT, gx); };
  auto shorter = [&](int k, int v) -> int {
    const int need = (v - 1) * kPfKeys - prefix[k] + 1;  // positions up to the tile's end
    if (need > q_len[k]) return tiles(k);
    return min(need > 0 ? (need + PT - 1) / PT - 1 : 0, tiles(k));
  };
  auto count = [&](int v) -> int {  // all tiles at least v long
    int c = 0;
#pragma unroll
    for (int k = 0; k < kSeqsPerLane; ++k)
      if (k < per) c += tiles(k) - shorter(k, v);
    return __reduce_add_sync(0xffffffffu, c);
  };
  WorkItem item{-1, 0, 0};
  const int rank = r / p.hkv;
  if (rank >= count(1)) return item;
  int lo = 1, hi = longest + 1;  // count(lo) > rank >= count(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (count(mid) > rank)
      lo = mid;
    else
      hi = mid;
  }
  // the item is among the tiles of length lo: its place there, (s, mt, g) order
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kSeqsPerLane; ++k)
    if (k < per) mine += shorter(k, lo + 1) - shorter(k, lo);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const int at = r - p.hkv * count(lo + 1);
  int j = at / p.hkv - (incl - mine);  // among the lane's own tiles
  const bool here = j >= 0 && j < mine;
  int s = 0, mt = 0;
#pragma unroll
  for (int k = 0; k < kSeqsPerLane; ++k)
    if (k < per && here && j >= 0) {
      const int first = shorter(k, lo), n = shorter(k, lo + 1) - first;
      if (j < n) {
        s = lane * per + k;
        mt = first + j;
      }
      j -= n;
    }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  item.s = __shfl_sync(0xffffffffu, s, src & 31);
  item.mt = __shfl_sync(0xffffffffu, mt, src & 31);
  item.g = at % p.hkv;
  if (src < 0) item.s = -1;
  return item;
}

// Dims of which the row of last key `limit` sees a NaN code that was taken out of
// its tile; `at` is the row's first output element.
__device__ __noinline__ void write_nan_dims(const PrefillQParams &p, uint32_t nan0, int limit,
                                            long long at) {
#pragma unroll 1
  for (int d = 0; d < kHeadDim; ++d) {
    if ((int)lds32(nan0 + 4 * d) > limit) continue;
    if (p.out_f32)
      static_cast<uint32_t *>(p.out)[at + d] = 0x7FC00000u;
    else
      static_cast<uint16_t *>(p.out)[at + d] = 0x7FC0u;
  }
}

template <int G>
__global__ void __launch_bounds__(kQpThreads, 2)
    prefill_fp8_block_kernel(const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ PrefillQParams p) {
  constexpr int PT = kPfRows / G;  // query positions per tile
  // always a programmatic dependent: it waits for the kernel before first of
  // all (and reads nothing by the read-only path), so only its set-up moves
  // ahead, about 2 us of a call behind another.  It does not let the next
  // kernel in early: CTAs that wait beside its own cost 2.5 % here
  griddep_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_addr(smem);
  uint64_t *slots = reinterpret_cast<uint64_t *>(smem + kQpOffBar);
  const uint32_t slot0 = smem_addr(slots);
  auto slot = [&](int i) { return slot0 + 8 * i; };
  const uint32_t b_s0 = slot(kSlS), b_p0 = slot(kSlP), b_o0 = slot(kSlO);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(slots + kSlTmem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slots + kSlAbort);

  const int tid = threadIdx.x, lane = tid & 31;
  // The warp's role.  Roles 0 .. 3 of the CTAs of every other round over the
  // SMs change places two by two, so that the widening warps of the two CTAs of
  // an SM (as a rule of neighbouring rounds) issue from different quarters of
  // it: 878 -> 869 us.
  const int place = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const unsigned linear = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
  const int warp = place < 4 ? place ^ (int)((linear / (unsigned)p.sms & 1u) << 1) : place;
  // the work item: longest first while a warp's lanes hold the sequences, else
  // in grid order with the last tiles of a chunk first
  int s, mt, g;
  if (p.num_seqs <= 32 * kSeqsPerLane) {
    const WorkItem item = pick_item<PT>(p, (int)gridDim.x, (int)linear);
    if (item.s < 0) return;
    s = item.s;
    mt = item.mt;
    g = item.g;
  } else {
    mt = (int)gridDim.x - 1 - (int)blockIdx.x;
    g = blockIdx.y;
    s = blockIdx.z;
    const int ql = p.cu_seqlens[s + 1] - p.cu_seqlens[s];
    if (mt == (int)gridDim.x - 1 && (unsigned)(mt * PT + PT) < (unsigned)ql && tid == 0)
      report(p.err, PA_DEVERR_SHAPE);  // rows past max_q_len: no CTA covers them
    if (mt * PT >= ql) return;
    if (p.context_lens[s] < ql) {
      if (tid == 0) report(p.err, PA_DEVERR_SHAPE);
      return;
    }
  }
  const int q0 = p.cu_seqlens[s];
  const int q_len = p.cu_seqlens[s + 1] - q0;
  const int pos0 = mt * PT;
  const int n = p.context_lens[s];
  const int prefix = n - q_len;
  const int npos = min(PT, q_len - pos0);
  // a chunk with rows outside q or a context longer than its table row: none of
  // the tile's rows is read or written (an early return here made the whole kernel
  // 8 % slower), and the keys end where the table row does
  const bool inside =
      q0 >= 0 && q0 + (long long)q_len <= p.total_tokens && n <= p.max_context;
  if (!inside && tid == 0) report(p.err, PA_DEVERR_SHAPE);
  const int rows = inside ? npos * G : 0;
  // last key any row of the tile sees
  const int kmax = min(prefix + pos0 + npos, p.max_context) - 1;
  const int nkv = kmax / kPfKeys + 1;

  if (tid == 0) {
    for (int i = 0; i < kQpKStages; ++i) {
      mbar_init(slot(kSlKFull + i), 1);
      mbar_init(slot(kSlKEmpty + i), 1);
    }
    for (int i = 0; i < kQpCStages; ++i) {
      mbar_init(slot(kSlCFull + i), 1);
      mbar_init(slot(kSlCEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(slot(kSlVFull + i), 1);
      mbar_init(slot(kSlVEmpty + i), 1);
      mbar_init(b_s0 + 8 * i, 1);
      mbar_init(b_p0 + 8 * i, kQpSoft / 32);
      mbar_init(b_o0 + 8 * i, 1);
    }
    mbar_init(slot(kSlQ), kQpSoft);
    for (int i = 0; i < 8; ++i) mbar_init(slot(kSlScale + i), 1);
    *abort_flag = 0;
    sts32(base + kQpOffNan - 4, 0u);
    fence_barrier_init();
  }
  if (tid < kHeadDim) sts32(base + kQpOffNan + 4 * tid, (uint32_t)INT_MAX);
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kQpTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + kQpTmemO;
  const int32_t *row = p.block_tables + (long long)s * p.bt_stride;

  if (warp == 0) {
    request_tiles(p, &tmap_k, row, n, nkv, g, base, slot0, abort_flag);
  } else if (warp == 2) {
    widen_v_tiles(p, n, nkv, prefix + pos0, base, slot0, abort_flag);
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers, each a whole converged warp: 1 issues S_j = Q K_j^T
    //      into buffer j & 1 once the PV of tile j - 2, which read that
    //      buffer, is done; 3 issues O += P'_j V_j ----
    constexpr uint32_t idesc_qk = idesc_format0(kPfKeys), idesc_pv = idesc_format0(kHeadDim);
    constexpr unsigned kAll = 0xffffffffu;
    uint32_t last_bar = 0;  // barrier of this warp's latest commit (drained on abort)
    int last_par = 0;
    if (warp == 1) {
      bool ok = __all_sync(kAll, mbar_wait_soon(slot(kSlQ), 0, abort_flag, p.err));
      tc_fence_after();
      for (int j = 0; j < nkv && ok; ++j) {
        const int b = j & 1, par = (j >> 1) & 1, ks = j % kQpKStages;
        ok = __all_sync(kAll, mbar_wait_soon(slot(kSlKFull + ks), (j / kQpKStages) & 1,
                                             abort_flag, p.err));
        if (ok && j >= 2)
          ok = __all_sync(kAll, mbar_wait_soon(b_o0 + 8 * b, par ^ 1, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
        issue_scores(tmem + b * kQpTmemS, umma_desc(base + kQpOffQ, 16, 1024),
                     umma_desc(base + kQpOffK + ks * kQpCodes, 16, 1024), idesc_qk, b_s0 + 8 * b,
                     slot(kSlKEmpty + ks));
        last_bar = b_s0 + 8 * b;
        last_par = par;
      }
    } else {
      for (int j = 0; j < nkv; ++j) {
        const int b = j & 1, par = (j >> 1) & 1;
        // (V first: it is there long before P', whose wait is the step's end)
        if (!__all_sync(kAll, mbar_wait_soon(slot(kSlVFull + b), par, abort_flag, p.err) &&
                                  mbar_wait_soon(b_p0 + 8 * b, par, abort_flag, p.err)))
          break;
        tc_fence_after();
        issue_values(tmem_o, tmem + b * kQpTmemS,
                     umma_desc(base + kQpOffV + b * kQpTile, 16, 1024), idesc_pv, j > 0,
                     b_o0 + 8 * b, slot(kSlVEmpty + b));
        last_bar = b_o0 + 8 * b;
        last_par = par;
      }
    }
    if (__any_sync(kAll, *abort_flag != 0) && last_bar) {
      // issued MMAs finish before TMEM is released (bounded)
      volatile int never = 0;
      mbar_wait(last_bar, last_par, &never, nullptr);
    }
    __syncwarp();
  } else {
    // ---- softmax: a row per thread (TMEM lane quarter warp % 4) ----
    const int lb = 32 * (warp & 3);
    const int r = lb + lane;
    const int rpos = r / G, hs = r % G;
    const bool rvalid = r < rows;
    const int limit = rvalid ? prefix + pos0 + rpos : -1;  // last key this row sees
    const uint32_t trow = (uint32_t)lb << 16;
    const long long orow = ((long long)(q0 + pos0 + rpos) * p.hq + g * G + hs) * kHeadDim;
    float c_row, bad = 0.f;  // factor of the row's scores; NaN for a row that is not finite
    {
      // the Q row as two E4M3 terms of q 2^-eq, in the K-major swizzled tiles
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + orow);
      uint4 qv[16];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        qv[c] = rvalid ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        uint32_t *w = &qv[c].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = (w[i] & p.q_and) ^ p.q_xor;
          const uint32_t a = w[i] & 0x7FFF7FFFu;
          top = max(top, max(a >> 16, a & 0xFFFFu));  // magnitudes order like their bits
        }
      }
      if (top >= 0x7F80u) bad = __uint_as_float(0x7FC00000u);
      const int eq = query_scale_for(__uint_as_float(top << 16));
      const float inv = inv_scale_of(eq);
      c_row = p.qk_scale_log2 * scale_of(eq);
#pragma unroll
      for (int c = 0; c < 8; ++c) {  // 16 dims
        const uint32_t w[8] = {qv[2 * c].x,     qv[2 * c].y,     qv[2 * c].z,     qv[2 * c].w,
                               qv[2 * c + 1].x, qv[2 * c + 1].y, qv[2 * c + 1].z, qv[2 * c + 1].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h[2], r2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = bf16x2_to_float2(w[2 * i + k]);
            const float x = f.x * inv, y = f.y * inv;
            h[k] = e4m3x2_of(x, y);
            const float2 v = codes_to_float2(h[k]);
            r2[k] = e4m3x2_of(x - v.x, y - v.y);
          }
          hi[i] = h[0] | (h[1] << 16);
          lo[i] = r2[0] | (r2[1] << 16);
        }
        sts128(base + kQpOffQ + sw128(r, c), hi[0], hi[1], hi[2], hi[3]);
        sts128(base + kQpOffQ + kQpQ + sw128(r, c), lo[0], lo[1], lo[2], lo[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(slot(kSlQ));
    }

    // m: the row's reference of t; it moves only when a tile's largest t
    // exceeds it by more than 8, so P' <= 256 and O is rescaled rarely
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nkv && ok; ++j) {
      const int b = j & 1, par = (j >> 1) & 1;
      ok = __all_sync(0xffffffffu,
                      mbar_wait_soon(slot(kSlScale + (j & 7)), (j >> 3) & 1, abort_flag, p.err) &&
                          mbar_wait_soon(b_s0 + 8 * b, par, abort_flag, p.err));
      const uint2 sc = lds64(slot(kSlScales + (j & 7)));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sb = tmem + b * kQpTmemS;
      const int key0 = j * kPfKeys;
      if (key0 + kPfKeys - 1 > prefix + pos0) {
        // a row may not see every key: those scores become -inf in place, out
        // of the way of the full tiles' instructions
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          uint32_t v[16];
          tmem_ld16(sb + trow + 16 * h, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = key0 + 16 * h + i <= limit ? v[i] : 0xFF800000u;
          tmem_st16(sb + trow + 16 * h, v);
          tmem_wait_st();
        }
      }
      float sv[2][32];
      tmem_ld64(sb + trow, sv);
      // per page: factor and offset of the exponent, the largest t
      float ck[kQpPages], ev[kQpPages], top = -INFINITY;
#pragma unroll
      for (int pg = 0; pg < kQpPages; ++pg) {
        // (at least the smallest normal: a masked -inf must stay -inf)
        ck[pg] = fmaxf(c_row * scale_of((sc.x >> (8 * pg)) & 0xFF), 1.17549435e-38f);
        ev[pg] = (float)((int)((sc.y >> (8 * pg)) & 0xFF) - kScaleBias);
        const float *x = &sv[pg >> 1][16 * (pg & 1)];
        const float a = fmax3(x[0], x[1], x[2]), c = fmax3(x[3], x[4], x[5]);
        const float d = fmax3(x[6], x[7], x[8]), e = fmax3(x[9], x[10], x[11]);
        const float f = fmax3(x[12], x[13], x[14]);
        const float mx = fmax3(fmax3(a, c, d), fmax3(e, f, x[15]), -INFINITY);
        top = fmaxf(top, fmaf(mx, ck[pg], ev[pg]));
      }
      const bool grow = top > m + 8.f;
      const float m_new = grow ? top : m;
      const float alpha = grow && m != -INFINITY ? exp2f(m - m_new) : 1.f;
      m = m_new;
      // rows whose reference moved rescale O, once the PV of tile j - 1 is
      // done and before that of tile j (tcgen05.ld / st are warp-collective)
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        if (j >= 1) {
          ok = __all_sync(0xffffffffu, mbar_wait_soon(b_o0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1,
                                                abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < kHeadDim / 32; ++c) {
          float ov[32];
          tmem_ld32(tmem_o + trow + c * 32, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] *= alpha;
          tmem_st32(tmem_o + trow + c * 32, ov);
        }
      }
      l *= alpha;
      // P' and the row sum, a page at a time.  A masked key has S = -inf and
      // 2^-inf = +0; a row with no key yet takes m = 0.
      const float neg_m = m == -INFINITY ? 0.f : -m;
#pragma unroll
      for (int pg = 0; pg < kQpPages; ++pg) {
        const float *x = &sv[pg >> 1][16 * (pg & 1)];
        const uint64_t c2 = pack_f32x2(ck[pg], ck[pg]);
        const float off = ev[pg] + neg_m + bad;
        const uint64_t o2 = pack_f32x2(off, off);
        uint64_t sum[2] = {0ull, 0ull};
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y0, y1;
          unpack_f32x2(fma_f32x2(pack_f32x2(x[2 * i], x[2 * i + 1]), c2, o2), y0, y1);
          const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
          sum[i & 1] = add_f32x2(sum[i & 1], pack_f32x2(e0, e1));
          h[i] = f16x2_of(e0, e1);
        }
        tmem_st8(sb + trow + pg * 8, h);
        float s0, s1;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
        l = fmaf(s0 + s1, inv_scale_of((sc.y >> (8 * pg)) & 0xFF), l);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_p0 + 8 * b);
    }
    // out = O / l
    if (ok && nkv > 0)
      ok = __all_sync(0xffffffffu, mbar_wait_soon(b_o0 + 8 * ((nkv - 1) & 1), ((nkv - 1) >> 1) & 1,
                                            abort_flag, p.err));
    tc_fence_after();
    if (ok) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int c = 0; c < kHeadDim / 32; ++c) {
        float ov[32];
        tmem_ld32(tmem_o + trow + c * 32, ov);
        if (!rvalid) continue;
        if (p.out_f32) {
          float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + orow + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(ov[4 * i] * inv, ov[4 * i + 1] * inv, ov[4 * i + 2] * inv,
                                 ov[4 * i + 3] * inv);
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + orow + c * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(float2_to_bf16x2(ov[8 * i] * inv, ov[8 * i + 1] * inv),
                                float2_to_bf16x2(ov[8 * i + 2] * inv, ov[8 * i + 3] * inv),
                                float2_to_bf16x2(ov[8 * i + 4] * inv, ov[8 * i + 5] * inv),
                                float2_to_bf16x2(ov[8 * i + 6] * inv, ov[8 * i + 7] * inv));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp >= 4 && lds32(base + kQpOffNan - 4)) {
    const int r = 32 * (warp & 3) + lane;
    if (r < rows)
      write_nan_dims(p, base + kQpOffNan, prefix + pos0 + r / G,
                     ((long long)(q0 + pos0 + r / G) * p.hq + g * G + r % G) * kHeadDim);
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kQpTmemCols)
                 : "memory");
  }
}

// (dim 128, kv head, token slot) view of the K pool; one box = 128 dims x 1
// head x 16 slots (one page of one head), 128-byte swizzle.
bool k_pool_map(CUtensorMap *map, const void *pool, long long num_blocks, int hkv) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)hkv, (cuuint64_t)num_blocks * kBlockSize};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)hkv * kHeadDim};
  cuuint32_t box[3] = {(cuuint32_t)kHeadDim, 1, (cuuint32_t)kBlockSize};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(pool), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G>
cudaError_t launch_prefill_q(const CUtensorMap &tk, const PrefillQParams &p, int max_q_len, cudaStream_t s, int device) {
  static std::atomic<bool> configured[64] = {};
  const cudaError_t e = set_smem_once(configured, prefill_fp8_block_kernel<G>, device, kQpSmem);
  if (e != cudaSuccess) return e;
  // two CTAs per SM: all of the unified L1 / shared memory as shared memory
  cudaFuncSetAttribute(prefill_fp8_block_kernel<G>, cudaFuncAttributePreferredSharedMemoryCarveout,
                       100);
  constexpr int PT = kPfRows / G;
  const dim3 grid((max_q_len + PT - 1) / PT, p.hkv, p.num_seqs);
  return launch_kernel(prefill_fp8_block_kernel<G>, grid, dim3(kQpThreads), kQpSmem, s, true, tk, p);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_prefill_fp8_block(
    void *out, int32_t out_dtype, const void *q, const int32_t *cu_seqlens, int32_t num_seqs,
    int32_t total_tokens, int32_t max_q_len, const void *k_cache, const void *v_cache,
    const uint8_t *k_scale, const uint8_t *v_scale, int64_t num_blocks,
    const int32_t *block_tables, int32_t block_table_stride, const int32_t *context_lens,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, float scale,
    int32_t *error_flags, void *stream) {
  using namespace pa;
  if (num_seqs < 0 || total_tokens < 0 || max_q_len < 0 || num_blocks < 0)
    return PA_ERR_INVALID_ARG;
  if (out_dtype != PA_DTYPE_BF16 && out_dtype != PA_DTYPE_F32) return PA_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (!(num_kv_heads == 1 || num_kv_heads == 2 || num_kv_heads == 4 || num_kv_heads == 8))
    return PA_ERR_UNSUPPORTED;
  if (num_q_heads < num_kv_heads || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 8)
    return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_tokens == 0 || max_q_len == 0) return PA_OK;
  if (num_seqs > 65535) return PA_ERR_UNSUPPORTED;
  if (num_blocks < 1 || num_blocks > (long long)(0x7fffffff / kBlockSize))
    return PA_ERR_INVALID_ARG;
  if (!out || !q || !cu_seqlens || !k_cache || !v_cache || !k_scale || !v_scale ||
      !block_tables || !context_lens)
    return PA_ERR_INVALID_ARG;
  if (block_table_stride < 1) return PA_ERR_INVALID_ARG;
  auto misaligned = [](const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15) != 0; };
  if (misaligned(out) || misaligned(q) || misaligned(k_cache) || misaligned(v_cache))
    return PA_ERR_INVALID_ARG;
  int device = -1, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
      sms < 1)
    return PA_ERR_DEVICE;
  CUtensorMap tk;
  memset(&tk, 0, sizeof tk);
  if (!k_pool_map(&tk, k_cache, num_blocks, num_kv_heads)) return PA_ERR_DEVICE;
  PrefillQParams p;
  p.out = out;
  p.out_f32 = out_dtype == PA_DTYPE_F32;
  p.q = static_cast<const uint16_t *>(q);
  p.cu_seqlens = cu_seqlens;
  p.num_seqs = num_seqs;
  p.total_tokens = total_tokens;
  p.sms = sms;
  p.v_cache = static_cast<const uint8_t *>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_blocks = num_blocks;
  p.block_tables = block_tables;
  p.bt_stride = block_table_stride;
  p.max_context = block_table_stride < INT_MAX / kBlockSize ? block_table_stride * kBlockSize
                                                            : INT_MAX;
  p.context_lens = context_lens;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  // the softmax takes maxima of raw scores and masks them before scaling,
  // which needs a positive scale: a negative one is folded into q (sign bits
  // flipped, exact), a zero one makes q zero
  p.qk_scale_log2 = (scale > 0.f ? scale : scale < 0.f ? -scale : 1.f) * 1.4426950408889634f;
  p.q_and = scale == 0.f ? 0u : 0xFFFFFFFFu;
  p.q_xor = scale < 0.f ? 0x80008000u : 0u;
  p.err = error_flags;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (num_q_heads / num_kv_heads) {
    case 1: e = launch_prefill_q<1>(tk, p, max_q_len, st, device); break;
    case 2: e = launch_prefill_q<2>(tk, p, max_q_len, st, device); break;
    case 3: e = launch_prefill_q<3>(tk, p, max_q_len, st, device); break;
    case 4: e = launch_prefill_q<4>(tk, p, max_q_len, st, device); break;
    case 5: e = launch_prefill_q<5>(tk, p, max_q_len, st, device); break;
    case 6: e = launch_prefill_q<6>(tk, p, max_q_len, st, device); break;
    case 7: e = launch_prefill_q<7>(tk, p, max_q_len, st, device); break;
    default: e = launch_prefill_q<8>(tk, p, max_q_len, st, device); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_LAUNCH;
}
