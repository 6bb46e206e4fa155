// pa_prefill_fp8_block: causal varlen attention of cu_seqlens-packed query
// chunks over a block-scaled FP8 cache (pa_fp8_block.cuh), on tcgen05.
//
// One CTA computes a 128-row tile of one (sequence, kv head), rows being the
// (query position, query head) pairs of 128 / G positions, over 64-key tiles:
//   S   = Q C_k^T        f16 x f16 -> fp32 (C: codes, exact in f16)
//   t   = c 2^ek S + ev  base-2 score plus the exponent of the key's V scale
//   P'  = 2^(t - m)      with m the row's running reference of t
//   O  += P' C_v         f16 x f16 -> fp32 in TMEM
//   l  += 2^-ev P'       per 16-key page;        out = O / l.
// Neither scale is applied to an element: K's goes into the page's constants
// of the exponent, V's into its offset, so P' <= 256 carries weight times V
// scale relative to the largest such product and one f16 term of it (11
// bits) suffices for a 4-bit significand.  That halves the PV products of a
// bf16 cache (whose weights take two bf16 terms) and its softmax's packing.
//
// Codes are widened on the way into shared memory by two converter warps (K,
// V), each with a rolling window of eight 16-byte loads per lane: a chunk is
// requested as soon as the one eight before it is converted, so half an 8 KB
// tile is always in flight per warp.  K pages (token-major)
// give K-major rows of the score MMA; V pages are dim-major, [128 dims][16
// tokens], which are K-major rows (a dim, 64 keys = 128 bytes) of the PV MMA
// with no transpose.  Both land in the 128-byte swizzle, and the lanes are
// laid over (row, chunk) so that a store instruction hits every bank once.
//
// Warps: 0 converts K, 2 converts V, 1 issues the score MMAs, 3 the PV MMAs,
// 4 .. 7 run the softmax, a row per thread.  Two CTAs share an SM: one's
// softmax runs while the other's MMAs use the tensor pipe.  A NaN or
// infinite value of q or of a key reaches every row of the tiles that meet
// it, those that do not attend to that key included (0 * NaN in the MMA).
#include <cmath>

#include "pa_fp8_block.cuh"
#include "pa_prefill_common.cuh"

namespace pa {
namespace {

constexpr int kQpThreads = 256;
constexpr int kQpSoft = 128;                    // softmax threads
constexpr int kQpPages = kPfKeys / kBlockSize;  // pages per KV tile
constexpr int kQpKHalf = kPfKeys * 128;         // 64 keys x 64 dims, f16
constexpr int kQpTile = 2 * kQpKHalf;           // one K or V tile, f16: 16 KB
constexpr int kQpQHalf = kPfRows * 128;         // 128 rows x 64 dims of Q
constexpr int kQpStages = 2;
constexpr int kQpAhead = 8;  // chunks a converter lane requests ahead (of 16 in a tile)
static_assert(16 % kQpAhead == 0, "a tile's chunks cycle through the window");
constexpr int kQpOffQ = 0;
constexpr int kQpOffK = kQpOffQ + 2 * kQpQHalf;
constexpr int kQpOffV = kQpOffK + kQpStages * kQpTile;
constexpr int kQpOffBar = kQpOffV + kQpStages * kQpTile;
// 8-byte slots: K full / empty, V full / empty (per stage), Q ready, two score,
// two P and two PV barriers, four scale barriers, TMEM address, abort flag;
// then the page scales of four tiles (K's four bytes, V's four)
constexpr int kSlKFull = 0, kSlKEmpty = 2, kSlVFull = 4, kSlVEmpty = 6, kSlQ = 8, kSlS = 9,
              kSlP = 11, kSlO = 13, kSlScale = 15, kSlTmem = 19, kSlAbort = 20, kSlScales = 21;
constexpr int kQpBarBytes = 256;
static_assert((kSlScales + 4) * 8 <= kQpBarBytes, "barrier slots do not fit");
constexpr int kQpSmem = 1024 + kQpOffBar + kQpBarBytes;
static_assert(kWorkOrderBytes <= kQpStages * kQpTile, "work-order scratch does not fit");
// TMEM (256 columns, two CTAs per SM): scores of tile j in buffer j % 2 at 0
// and 64, P' over the scores it came from (32 columns, two keys each), O at 128
constexpr int kQpTmemCols = 256, kQpTmemS = 64, kQpTmemO = 128;

struct PrefillQParams {
  void *out;
  int out_f32;
  const uint16_t *q;
  const int32_t *cu_seqlens;
  int num_seqs;
  const uint8_t *k_cache, *v_cache;
  const uint8_t *k_scale, *v_scale;
  long long num_blocks;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int hq, hkv;
  float qk_scale_log2;    // > 0: a scale <= 0 is folded into q as staged
  uint32_t q_and, q_xor;  // staged q pairs = (q & q_and) ^ q_xor
  int32_t *err;
};

// Instruction descriptor, kind::f16: f16 A and B (both K-major), fp32 D, M =
// 128, N = n.
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kPfRows >> 4) << 24);
}

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
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// A converter warp's stream of 64-key tiles of K (or V) of one (sequence, kv
// head).  Chunk i of a tile (16 codes per lane) belongs to page i / 4 of the
// tile; a page is four chunks: K token rows 4 (i % 4) .. + 3, or V dims
// 32 (i % 4) .. + 31.  Pages with no key, and bad entries, read as zero codes.
template <bool kIsV>
__device__ __forceinline__ void convert_tiles(const PrefillQParams &p, const int32_t *row, int n,
                                              int nkv, int g, uint32_t dst0, uint32_t b_full0,
                                              uint32_t b_empty0, uint32_t b_scale0,
                                              uint32_t scales0, volatile int *abort_flag) {
  const int lane = threadIdx.x & 31;
  // the lane's place in a chunk: K (row, 16-dim group), two rows and four
  // groups per quarter warp; V dim row = lane
  const int kr = ((lane >> 2) & 1) + 2 * (lane >> 4), kc = (lane & 3) + 4 * ((lane >> 3) & 1);
  const long long row_bytes = (long long)p.hkv * kHeadDim;
  const uint8_t *pool = kIsV ? p.v_cache + (long long)g * (kHeadDim * kBlockSize) + lane * kBlockSize
                             : p.k_cache + (long long)g * kHeadDim + kr * row_bytes + kc * 16;
  const long long page_bytes = row_bytes * kBlockSize;
  const long long sub_bytes = kIsV ? 32 * kBlockSize : 4 * row_bytes;

  // table entries of eight tiles (32 pages) per round of lane loads, the next
  // round requested a tile ahead of its first use; -1: nothing to read
  auto entries = [&](int j8) -> int {
    const int lb = j8 * 32 + lane;
    if (lb * kBlockSize >= n) return -1;
    const int ph = lb < p.bt_stride ? __ldg(row + lb) : -1;
    const bool ok = ph >= 0 && ph < p.num_blocks;
    if (!ok && !kIsV) report(p.err, PA_DEVERR_BLOCK_INDEX);
    return ok ? ph : -1;
  };
  int round = entries(0);
  uint4 buf[kQpAhead];
  uint32_t scale = 0;  // lane pg < 4: scale byte of page pg of the tile in buf (K warp: V's << 8)
  int now[kQpPages], next[kQpPages];  // pages of tile j and of the one after it
  auto load_scales = [&](int j) {
    if constexpr (!kIsV) {
      // both scales of the page, by the K warp (it feeds the softmax first)
      const int ph = __shfl_sync(0xffffffffu, round, (j & 7) * kQpPages + (lane & 3));
      scale = (uint32_t)kScaleBias * 0x101u;
      if (lane < kQpPages && ph >= 0)
        scale = (uint32_t)__ldg(p.k_scale + (long long)ph * p.hkv + g) |
                ((uint32_t)__ldg(p.v_scale + (long long)ph * p.hkv + g) << 8);
    }
  };
  auto pages_of = [&](int j) {
#pragma unroll
    for (int pg = 0; pg < kQpPages; ++pg) {
      now[pg] = next[pg];
      next[pg] = __shfl_sync(0xffffffffu, round, (j & 7) * kQpPages + pg);
    }
  };
  // chunk i of the tile whose pages are now (i < 16) or next
  auto load = [&](int i) {
    const int ph = i < 16 ? now[i >> 2] : next[(i - 16) >> 2];
    buf[i % kQpAhead] = ph >= 0 ? __ldg(reinterpret_cast<const uint4 *>(pool + ph * page_bytes +
                                                             (i & 3) * sub_bytes))
                     : make_uint4(0u, 0u, 0u, 0u);
  };
#pragma unroll
  for (int pg = 0; pg < kQpPages; ++pg) next[pg] = -1;
  pages_of(0);
  load_scales(0);
#pragma unroll
  for (int i = 0; i < kQpAhead; ++i) load(16 + i);

  for (int j = 0; j < nkv; ++j) {
    const int st = j & 1;
    const bool more = j + 1 < nkv;
    const uint32_t mine = scale;
    if (more && ((j + 1) & 7) == 0) round = entries((j + 1) >> 3);
    pages_of(j + 1);  // (past the last tile: loads nothing)
    if (more) load_scales(j + 1);
    if (j >= 2 && !__all_sync(0xffffffffu, mbar_wait(b_empty0 + 8 * st, ((j >> 1) - 1) & 1,
                                                     abort_flag, p.err)))
      return;
    if constexpr (!kIsV) {
      // the scales of tile j: slot j % 4, last read by the softmax of tile
      // j - 4, which is over: the score MMA of tile j - 2 waited for its PV
      const uint32_t c = clamp_scales4(mine & 0xFFFFu);
      if (lane < kQpPages) {
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales0 + 8 * (j & 3) + lane), "r"(c & 0xFFu)
                     : "memory");
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales0 + 8 * (j & 3) + 4 + lane),
                     "r"((c >> 8) & 0xFFu)
                     : "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_scale0 + 8 * (j & 3));
    }
    const uint32_t dst = dst0 + st * kQpTile;
    const int key0 = j * kPfKeys;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint4 w = buf[i % kQpAhead];
      if (i + kQpAhead < 16 || more) load(i + kQpAhead);
      if constexpr (kIsV) {
        // tokens past the last key weigh 0 and may hold anything: zero codes
        const int left = n - (key0 + (i >> 2) * kBlockSize);
        if (left < kBlockSize) {
          uint32_t *x = &w.x;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int keep = min(max(left - 4 * q, 0), 4);
            x[q] &= keep >= 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
          }
        }
      }
      const uint32_t a0 = f16x2_of_codes(w.x), a1 = f16x2_of_codes(w.x >> 16);
      const uint32_t a2 = f16x2_of_codes(w.y), a3 = f16x2_of_codes(w.y >> 16);
      const uint32_t b0 = f16x2_of_codes(w.z), b1 = f16x2_of_codes(w.z >> 16);
      const uint32_t b2 = f16x2_of_codes(w.w), b3 = f16x2_of_codes(w.w >> 16);
      uint32_t at;
      int r, c;
      if constexpr (kIsV) {
        r = 32 * (i & 3) + lane;  // dim
        c = 2 * (i >> 2);         // its 16 tokens: two 16-byte chunks
        at = dst;
      } else {
        r = 16 * (i >> 2) + 4 * (i & 3) + kr;  // key
        c = 2 * (kc & 3);
        at = dst + (kc >> 2) * kQpKHalf;
      }
      sts128(at + sw128(r, c), a0, a1, a2, a3);
      sts128(at + sw128(r, c + 1), b0, b1, b2, b3);
    }
    // visible to the tensor core before the tile is handed over
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    mbar_arrive(b_full0 + 8 * st);
  }
}

template <int G>
__global__ void __launch_bounds__(kQpThreads, 2)
    prefill_fp8_block_kernel(const __grid_constant__ PrefillQParams p) {
  constexpr int PT = kPfRows / G;  // query positions per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_addr(smem);
  uint64_t *slots = reinterpret_cast<uint64_t *>(smem + kQpOffBar);
  auto slot = [&](int i) { return smem_addr(slots + i); };
  const uint32_t b_k_full0 = slot(kSlKFull), b_k_empty0 = slot(kSlKEmpty);
  const uint32_t b_v_full0 = slot(kSlVFull), b_v_empty0 = slot(kSlVEmpty);
  const uint32_t b_q = slot(kSlQ), b_s0 = slot(kSlS), b_p0 = slot(kSlP), b_o0 = slot(kSlO);
  const uint32_t b_scale0 = slot(kSlScale), scales0 = slot(kSlScales);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(slots + kSlTmem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(slots + kSlAbort);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // the work item: longest first while one thread per sequence suffices,
  // else in grid order with the last tiles of a chunk first
  int s, mt, g;
  if (p.num_seqs <= kQpThreads) {
    if (!pick_work_item<PT, kQpThreads>(p, (int)gridDim.x,
                                        reinterpret_cast<int *>(smem + kQpOffK), s, mt, g))
      return;
  } else {
    mt = (int)gridDim.x - 1 - (int)blockIdx.x;
    g = blockIdx.y;
    s = blockIdx.z;
    const int ql = __ldg(p.cu_seqlens + s + 1) - __ldg(p.cu_seqlens + s);
    if (mt == (int)gridDim.x - 1 && mt * PT + PT < ql && tid == 0)
      report(p.err, PA_DEVERR_SHAPE);  // rows past max_q_len: no CTA covers them
    if (mt * PT >= ql) return;
    if (__ldg(p.context_lens + s) < ql) {
      if (tid == 0) report(p.err, PA_DEVERR_SHAPE);
      return;
    }
  }
  const int q0 = __ldg(p.cu_seqlens + s);
  const int q_len = __ldg(p.cu_seqlens + s + 1) - q0;
  const int pos0 = mt * PT;
  const int n = __ldg(p.context_lens + s);
  const int prefix = n - q_len;
  const int npos = min(PT, q_len - pos0);
  const int rows = npos * G;
  const int kmax = prefix + pos0 + npos - 1;  // last key any row of the tile sees
  const int nkv = kmax / kPfKeys + 1;

  if (tid == 0) {
    for (int i = 0; i < kQpStages; ++i) {
      mbar_init(b_k_full0 + 8 * i, 32);
      mbar_init(b_k_empty0 + 8 * i, 1);
      mbar_init(b_v_full0 + 8 * i, 32);
      mbar_init(b_v_empty0 + 8 * i, 1);
      mbar_init(b_s0 + 8 * i, 1);
      mbar_init(b_p0 + 8 * i, kQpSoft);
      mbar_init(b_o0 + 8 * i, 1);
    }
    mbar_init(b_q, kQpSoft);
    for (int i = 0; i < 4; ++i) mbar_init(b_scale0 + 8 * i, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
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
    convert_tiles<false>(p, row, n, nkv, g, base + kQpOffK, b_k_full0, b_k_empty0, b_scale0,
                         scales0, abort_flag);
  } else if (warp == 2) {
    convert_tiles<true>(p, row, n, nkv, g, base + kQpOffV, b_v_full0, b_v_empty0, 0u, 0u,
                        abort_flag);
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers, each a whole converged warp: 1 issues S_j = Q K_j^T
    //      into buffer j & 1 once the PV of tile j - 2, which read that
    //      buffer, is done; 3 issues O += P'_j V_j ----
    constexpr uint32_t idesc_qk = idesc_f16(kPfKeys), idesc_pv = idesc_f16(kHeadDim);
    constexpr unsigned kAll = 0xffffffffu;
    uint32_t last_bar = 0;  // barrier of this warp's latest commit (drained on abort)
    int last_par = 0;
    if (warp == 1) {
      bool ok = __all_sync(kAll, mbar_wait(b_q, 0, abort_flag, p.err));
      tc_fence_after();
      for (int j = 0; j < nkv && ok; ++j) {
        const int b = j & 1, par = (j >> 1) & 1;
        ok = __all_sync(kAll, mbar_wait(b_k_full0 + 8 * b, par, abort_flag, p.err));
        if (ok && j >= 2)
          ok = __all_sync(kAll, mbar_wait(b_o0 + 8 * b, par ^ 1, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          umma_f16_ss(
              tmem + b * kQpTmemS,
              umma_desc(base + kQpOffQ + (ks >> 2) * kQpQHalf + (ks & 3) * 32, 16, 1024),
              umma_desc(base + kQpOffK + b * kQpTile + (ks >> 2) * kQpKHalf + (ks & 3) * 32, 16,
                        1024),
              idesc_qk, ks > 0);
        umma_commit(b_s0 + 8 * b);
        umma_commit(b_k_empty0 + 8 * b);
        last_bar = b_s0 + 8 * b;
        last_par = par;
      }
    } else {
      for (int j = 0; j < nkv; ++j) {
        const int b = j & 1, par = (j >> 1) & 1;
        if (!__all_sync(kAll, mbar_wait(b_p0 + 8 * b, par, abort_flag, p.err))) break;
        if (!__all_sync(kAll, mbar_wait(b_v_full0 + 8 * b, par, abort_flag, p.err))) break;
        tc_fence_after();
        // 4 k-steps of 16 keys: 32 bytes of every 128-byte dim row
#pragma unroll
        for (int ks = 0; ks < kPfKeys / 16; ++ks)
          umma_f16_ta(tmem_o, tmem + b * kQpTmemS + ks * 8,
                      umma_desc(base + kQpOffV + b * kQpTile + ks * 32, 16, 1024), idesc_pv,
                      (j > 0 || ks > 0) ? 1u : 0u);
        umma_commit(b_o0 + 8 * b);
        umma_commit(b_v_empty0 + 8 * b);
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
    {
      // the Q row, rounded to f16, into the K-major swizzled tile
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + orow);
      uint4 qv[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) qv[c] = rvalid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint32_t w[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2((w[i] & p.q_and) ^ p.q_xor);
          h[i] = f16x2_of(f.x, f.y);
        }
        sts128(base + kQpOffQ + (c >> 3) * kQpQHalf + sw128(r, c & 7), h[0], h[1], h[2], h[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(b_q);
    }

    // m: the row's reference of t; it moves only when a tile's largest t
    // exceeds it by more than 8, so P' <= 256 and O is rescaled rarely
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nkv && ok; ++j) {
      const int b = j & 1, par = (j >> 1) & 1;
      ok = __all_sync(0xffffffffu,
                      mbar_wait(b_scale0 + 8 * (j & 3), (j >> 2) & 1, abort_flag, p.err) &&
                          mbar_wait(b_s0 + 8 * b, par, abort_flag, p.err));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sb = tmem + b * kQpTmemS;
      const int key0 = j * kPfKeys;
      const uint2 sc = lds64(scales0 + 8 * (j & 3));
      float sv[2][32];
      tmem_ld64(sb + trow, sv);
      if (key0 + kPfKeys - 1 > prefix + pos0) {  // a row may not see every key
#pragma unroll
        for (int i = 0; i < kPfKeys; ++i)
          sv[i >> 5][i & 31] = key0 + i <= limit ? sv[i >> 5][i & 31] : -INFINITY;
      }
      // per page: factor and offset of the exponent, the largest t
      float ck[kQpPages], ev[kQpPages], top = -INFINITY;
#pragma unroll
      for (int pg = 0; pg < kQpPages; ++pg) {
        // (at least the smallest normal: a masked -inf must stay -inf)
        ck[pg] = fmaxf(p.qk_scale_log2 * scale_of((sc.x >> (8 * pg)) & 0xFF), 1.17549435e-38f);
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
          ok = __all_sync(0xffffffffu, mbar_wait(b_o0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1,
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
        const float off = ev[pg] + neg_m;
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
      mbar_arrive(b_p0 + 8 * b);
    }
    // out = O / l
    if (ok && nkv > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(b_o0 + 8 * ((nkv - 1) & 1), ((nkv - 1) >> 1) & 1,
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
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kQpTmemCols)
                 : "memory");
  }
}

template <int G>
cudaError_t launch_prefill_q(const PrefillQParams &p, int max_q_len, cudaStream_t s, int device) {
  static std::atomic<bool> configured[64] = {};
  const cudaError_t e = set_smem_once(configured, prefill_fp8_block_kernel<G>, device, kQpSmem);
  if (e != cudaSuccess) return e;
  // two CTAs per SM: all of the unified L1 / shared memory as shared memory
  cudaFuncSetAttribute(prefill_fp8_block_kernel<G>, cudaFuncAttributePreferredSharedMemoryCarveout,
                       100);
  constexpr int PT = kPfRows / G;
  const dim3 grid((max_q_len + PT - 1) / PT, p.hkv, p.num_seqs);
  return launch_kernel(prefill_fp8_block_kernel<G>, grid, dim3(kQpThreads), kQpSmem, s, false, p);
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
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_DEVICE;
  PrefillQParams p;
  p.out = out;
  p.out_f32 = out_dtype == PA_DTYPE_F32;
  p.q = static_cast<const uint16_t *>(q);
  p.cu_seqlens = cu_seqlens;
  p.num_seqs = num_seqs;
  p.k_cache = static_cast<const uint8_t *>(k_cache);
  p.v_cache = static_cast<const uint8_t *>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_blocks = num_blocks;
  p.block_tables = block_tables;
  p.bt_stride = block_table_stride;
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
    case 1: e = launch_prefill_q<1>(p, max_q_len, st, device); break;
    case 2: e = launch_prefill_q<2>(p, max_q_len, st, device); break;
    case 3: e = launch_prefill_q<3>(p, max_q_len, st, device); break;
    case 4: e = launch_prefill_q<4>(p, max_q_len, st, device); break;
    case 5: e = launch_prefill_q<5>(p, max_q_len, st, device); break;
    case 6: e = launch_prefill_q<6>(p, max_q_len, st, device); break;
    case 7: e = launch_prefill_q<7>(p, max_q_len, st, device); break;
    default: e = launch_prefill_q<8>(p, max_q_len, st, device); break;
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_LAUNCH;
}
