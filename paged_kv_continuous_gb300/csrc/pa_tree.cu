// pa_decode_tree: attention of trees of drafted tokens over the paged bf16
// cache.  Node i of a sequence with P committed keys sees keys 0 .. P - 1 and
// the nodes on its way to the root (keys P + a), so with rows (node, head)
//   S = Q K^T,  P = exp2(c S - m) where seen,  O = P V,  l = sum P,  out = O / l
// and every key is read once for all the nodes and all the G query heads of its
// kv head.
//
// A unit is a 128-row tile of one (sequence, kv head); its keys are cut into
// 64-key tiles.  All units' tiles form one list (sequence, kv head, row tile),
// which is cut evenly over the CTAs, two per SM: a CTA runs the last tiles of
// one unit, some whole units and the first tiles of another.  A unit in one
// piece is written to `out`; the pieces of a cut one leave (O / l, m + log2 l)
// in the workspace, and tree_merge_kernel joins them.
//
// Roles of the 8 warps: 0 loads K tiles and 2 V tiles (TMA, two stages each),
// 1 issues the score MMAs and owns the tensor memory (two score buffers of 64
// columns, O in 128), 3 issues the PV MMAs with P from tensor memory, 4 .. 7 run
// the softmax, a row per thread, and write the rows.  They walk the list of
// pieces independently; the stages and buffers run on across pieces.
//
// A piece's tiles run from the last key to the first, so that a row finds the
// nodes it sees by one walk up its parents, which goes on where the tile before
// left it: no mask is ever stored, and the tree may have any size.
//
// P is kept as two bf16 terms, hi the truncated weight and lo the rounded rest
// (together 16 bits), each with its PV MMA: one term's error (2^-9 of a weight)
// is as large as the output's own rounding.
#include <climits>
#include <cmath>
#include <cstring>

#include "pa_prefill_common.cuh"

namespace pa {
namespace {

constexpr int kTrThreads = 256;
constexpr int kTrPages = kPfKeys / kBlockSize;  // pages per KV tile
constexpr int kTrHalf = kPfKeys * 128;          // 64 keys x 64 dims, 128-byte swizzle
constexpr int kTrTile = 2 * kTrHalf;            // one K or V tile
constexpr int kTrQHalf = kPfRows * 128;         // 128 rows x 64 dims of Q
constexpr int kTrStages = 2;
constexpr int kTrOffQ = 0;
constexpr int kTrOffK = kTrOffQ + 2 * kTrQHalf;
constexpr int kTrOffV = kTrOffK + kTrStages * kTrTile;
constexpr int kTrOffBar = kTrOffV + kTrStages * kTrTile;
// 8-byte slots: K full / empty and V full / empty per stage, Q, two score, two
// P and two PV barriers, the TMEM address, the abort flag, the last piece with
// a V row that is not finite
constexpr int kTsKFull = 0, kTsKEmpty = kTsKFull + kTrStages, kTsVFull = kTsKEmpty + kTrStages;
constexpr int kTsVEmpty = kTsVFull + kTrStages, kTsQ = kTsVEmpty + kTrStages, kTsS = kTsQ + 1;
constexpr int kTsP = kTsS + 2, kTsO = kTsP + 2, kTsTmem = kTsO + 2, kTsAbort = kTsTmem + 1;
constexpr int kTsBad = kTsAbort + 1, kTsSlots = 32;
static_assert(kTsBad < kTsSlots, "barrier slots do not fit");
constexpr int kTrSmem = 1024 + kTrOffBar + kTsSlots * 8;
static_assert(2 * (kTrSmem + 1024) <= 228 * 1024, "two CTAs do not fit an SM");
constexpr int kTrCols = 256;    // tensor memory columns: S_0 0.., S_1 64.., O 128..
constexpr int kTrSCols = 64, kTrO = 128;

// A piece's start and end cost about as much as this many tiles.
constexpr int kTrPieceTiles = 2;
// CTAs in use: none is given less than this many tiles.
constexpr int kTrMinTiles = 4;

struct TreeParams {
  void *out;
  int out_f32;
  const uint16_t *q;
  const int32_t *cu, *parents;
  int num_seqs, total_tokens, max_q_len;
  const uint16_t *v_cache;
  long long num_blocks;
  const int32_t *tables;
  long long bt_stride;
  const int32_t *ctx;
  int hq, hkv, group;
  float scale_log2;       // > 0: a scale <= 0 is folded into q as staged
  uint32_t q_and, q_xor;  // staged q pairs = (q & q_and) ^ q_xor
  int splits;             // CTAs of the launch
  int all_splits;         // use them all
  float *part_o;          // [2][splits][128 rows][128]
  float *part_lse;        // [2][splits][128]
  int32_t *err;
};

// ---- the list of tiles --------------------------------------------------------

struct TreeSeq {
  int q0, nodes, keys;  // nodes = 0: nothing to do
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int s, bool tell) {
  TreeSeq r;
  r.q0 = p.cu[s];
  const int end = p.cu[s + 1];
  r.keys = p.ctx[s];
  r.nodes = 0;
  if (end == r.q0) return r;
  // (differences in 64 bits: any int32 values)
  const long long n = (long long)end - r.q0;
  const bool ok = r.q0 >= 0 && end <= p.total_tokens && n > 0 && n <= p.max_q_len &&
                  n <= r.keys && ceil_div_blocks(r.keys) <= p.bt_stride;
  if (ok)
    r.nodes = (int)n;
  else if (tell)
    report(p.err, PA_DEVERR_SHAPE);
  return r;
}

// Tiles of row tile mt: up to the key of its last node.
__device__ __forceinline__ int unit_tiles(const TreeSeq &q, int group, int mt) {
  const int last = (min((mt + 1) * kPfRows, q.nodes * group) - 1) / group;
  return (q.keys - q.nodes + last) / kPfKeys + 1;
}
__device__ __forceinline__ int row_tiles(const TreeSeq &q, int group) {
  return (q.nodes * group + kPfRows - 1) / kPfRows;
}
// Length of one kv head of the sequence in the list.
__device__ __forceinline__ long long head_weight(const TreeSeq &q, int group) {
  long long w = 0;
  const int m = row_tiles(q, group);
  for (int i = 0; i < m; ++i) w += unit_tiles(q, group, i) + kTrPieceTiles;
  return w;
}

__device__ __forceinline__ long long ctas_in_use(const TreeParams &p, long long N) {
  if (N == 0) return 0;
  const long long most = p.all_splits ? N : N / (kTrMinTiles + kTrPieceTiles);
  return max(1ll, min((long long)p.splits, most));
}
__device__ __forceinline__ long long cta_begin(long long c, long long C, long long N) {
  return c * N / C;
}
// The CTA that holds place x: the largest c with cta_begin(c) <= x (C <= N).
__device__ __forceinline__ long long cta_of(long long x, long long C, long long N) {
  return ((x + 1) * C - 1) / N;
}

// Sums of a long long over the block: the total, and what lies before this thread.
__device__ __forceinline__ long long block_before(long long v, long long *warp_sum,
                                                  long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  long long before = x - v;
  total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  return before;
}

// A CTA's place in the list: the unit it is in and where that unit starts.
struct TreePlace {
  long long x, end, start;
  int s, g, mt;
};

struct TreePiece {
  TreeSeq q;
  int s, g, mt, t0, t1, tiles;
};

// The next piece of a CTA's part of the list; every warp runs this for itself.
struct TreeWalk {
  TreePlace at;
  TreeSeq q;

  __device__ __forceinline__ void begin(const TreeParams &p, const TreePlace &place) {
    at = place;
    q = tree_seq(p, at.s, false);
  }
  __device__ __forceinline__ bool next(const TreeParams &p, TreePiece &r) {
    while (at.x < at.end) {
      const int tiles = unit_tiles(q, p.group, at.mt);
      const long long rel = at.x - at.start;
      const bool got = rel < tiles;
      if (got) {
        r.q = q;
        r.s = at.s;
        r.g = at.g;
        r.mt = at.mt;
        r.tiles = tiles;
        r.t0 = (int)rel;
        r.t1 = (int)min((long long)tiles, at.end - at.start);
      }
      at.start += tiles + kTrPieceTiles;
      at.x = at.start;
      if (++at.mt == row_tiles(q, p.group)) {
        at.mt = 0;
        if (++at.g == p.hkv) {
          at.g = 0;
          if (at.x < at.end) do {
              q = tree_seq(p, ++at.s, false);
            } while (q.nodes == 0 && at.s + 1 < p.num_seqs);
        }
      }
      if (got) return true;
    }
    return false;
  }
};

// Finds the place of list position x0 (one thread of the block holds it) and the
// list's length.
__device__ __forceinline__ void tree_plan(const TreeParams &p, long long c, long long *warp_sum,
                                          TreePlace *place, long long &C, bool tell) {
  const int per = (p.num_seqs + (int)blockDim.x - 1) / (int)blockDim.x;
  const int s0 = min(p.num_seqs, (int)threadIdx.x * per), s1 = min(p.num_seqs, s0 + per);
  long long mine = 0, N;
  for (int s = s0; s < s1; ++s)
    mine += head_weight(tree_seq(p, s, tell), p.group) * p.hkv;
  long long before = block_before(mine, warp_sum, N);
  C = ctas_in_use(p, N);
  if (c >= C) return;
  const long long x0 = cta_begin(c, C, N);
  if (x0 < before || x0 >= before + mine) return;
  for (int s = s0; s < s1; ++s) {
    const TreeSeq q = tree_seq(p, s, false);
    const long long w = head_weight(q, p.group);
    if (x0 < before + w * p.hkv) {
      TreePlace r;
      r.x = x0;
      r.end = cta_begin(c + 1, C, N);
      r.s = s;
      r.g = (int)((x0 - before) / w);
      r.start = before + r.g * w;
      r.mt = 0;
      while (true) {
        const int len = unit_tiles(q, p.group, r.mt) + kTrPieceTiles;
        if (x0 < r.start + len) break;
        r.start += len;
        ++r.mt;
      }
      *place = r;
      return;
    }
    before += w * p.hkv;
  }
}

// ---- attention ----------------------------------------------------------------

// Of dims 32 cc .. 32 cc + 31, those where a drafted node that `node` sees in
// this piece has a V element that is not finite: the row is NaN there (the tile's
// copy was cleared, since 0 * NaN is NaN in the MMA).  Rare and slow.
__device__ __noinline__ uint32_t not_finite(const TreeParams &p, int s, int q0, int done, int g,
                                            int node, int first_key, int end_key, int cc) {
  const int32_t *par = p.parents + q0;
  uint32_t dims = 0;
  for (int a = node; a >= 0;) {
    const int key = done + a;
    if (key < first_key) break;
    if (key <= end_key) {
      const long long ph = p.tables[(long long)s * p.bt_stride + key / kBlockSize];
      if (ph >= 0 && ph < p.num_blocks) {
        const uint16_t *v =
            p.v_cache + ((ph * kBlockSize + key % kBlockSize) * p.hkv + g) * kHeadDim + cc * 32;
        for (int i = 0; i < 32; ++i)
          if ((v[i] & 0x7f80) == 0x7f80) dims |= 1u << i;
      }
    }
    const int up = par[a];
    a = up < a ? up : -1;
  }
  return dims;
}

__global__ void __launch_bounds__(kTrThreads, 2)
    tree_kernel(const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_addr(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kTrOffBar);
  const uint32_t b_k_full = smem_addr(bars + kTsKFull), b_k_empty = smem_addr(bars + kTsKEmpty);
  const uint32_t b_v_full = smem_addr(bars + kTsVFull), b_v_empty = smem_addr(bars + kTsVEmpty);
  const uint32_t b_q = smem_addr(bars + kTsQ), b_s = smem_addr(bars + kTsS);
  const uint32_t b_p = smem_addr(bars + kTsP), b_o = smem_addr(bars + kTsO);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kTsTmem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kTsAbort);
  volatile int *bad_piece = reinterpret_cast<volatile int *>(bars + kTsBad);
  __shared__ long long warp_sum[kTrThreads / 32];
  __shared__ TreePlace place;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kTrStages; ++i) {
      mbar_init(b_k_full + 8 * i, 1);
      mbar_init(b_k_empty + 8 * i, 1);
      mbar_init(b_v_full + 8 * i, 1);
      mbar_init(b_v_empty + 8 * i, 1);
    }
    mbar_init(b_q, kPfRows);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, kPfRows);
      mbar_init(b_o + 8 * i, 1);
    }
    *abort_flag = 0;
    *bad_piece = -1;
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
  }
  griddep_wait();
  griddep_launch_dependents();
  long long C;
  tree_plan(p, blockIdx.x, warp_sum, &place, C, blockIdx.x == 0);
  if ((long long)blockIdx.x >= C) return;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTrCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + kTrO;
  constexpr unsigned kAll = 0xffffffffu;

  TreeWalk walk;
  TreePiece u;
  walk.begin(p, place);
  // tiles done so far, over all pieces: their stage is it % 2, their score buffer too
  int it = 0;

  if (warp == 0 || warp == 2) {
    // ---- loaders: a tile's pages (64 dims x 16 keys a box) into stage it % 2
    //      once the MMAs that read its previous tile are done
    const bool is_k = warp == 0;
    const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
    const uint32_t dst0 = base + (is_k ? kTrOffK : kTrOffV);
    const uint32_t full0 = is_k ? b_k_full : b_v_full, empty0 = is_k ? b_k_empty : b_v_empty;
    bool ok = true;
    while (ok && walk.next(p, u)) {
      const int32_t *row = p.tables + (long long)u.s * p.bt_stride;
      // table entries of eight tiles, one per lane: -1 no key in the page
      // (left as it is: masked), -2 a bad entry
      int ph_lane = -1;
      for (int j = u.t1 - 1; j >= u.t0; --j, ++it) {
        const int st = it % kTrStages, round = it / kTrStages;
        if (j == u.t1 - 1 || j % (32 / kTrPages) == 32 / kTrPages - 1) {
          const long long page = (long long)(j / (32 / kTrPages)) * 32 + lane;
          const bool has = page * kBlockSize < u.q.keys;
          const int ph = has ? row[page] : -1;
          ph_lane = !has ? -1 : ph >= 0 && ph < p.num_blocks ? ph : -2;
        }
        if (round > 0 &&
            !__all_sync(kAll, mbar_wait(empty0 + 8 * st, (round - 1) & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        const int at = (j % (32 / kTrPages)) * kTrPages;
        const int phys = __shfl_sync(kAll, ph_lane, at + lane % kTrPages);
        const unsigned okm = __ballot_sync(kAll, lane < kTrPages && phys >= 0);
        if (__any_sync(kAll, phys == -2) && lane == 0) report(p.err, PA_DEVERR_BLOCK_INDEX);
        const uint32_t full = full0 + 8 * st;
        if (lane == 0) mbar_arrive_expect_tx(full, __popc(okm) * 2u * kBlockSize * 64 * 2);
        __syncwarp();
#pragma unroll
        for (int pg = 0; pg < kTrPages; ++pg) {
          if (!((okm >> pg) & 1u)) continue;
          const int z = __shfl_sync(kAll, ph_lane, at + pg) * kBlockSize;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_3d(dst0 + st * kTrTile + h * kTrHalf + pg * kBlockSize * 128, map, h * 64,
                        u.g, z, full);
        }
      }
    }
    if (lane == 0 && *abort_flag) {
      // copies in flight must land before the CTA's shared memory is released
      volatile int never = 0;
      for (int i = it > kTrStages ? it - kTrStages : 0; i < it; ++i)
        mbar_wait(full0 + 8 * (i % kTrStages), (i / kTrStages) & 1, &never, nullptr);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers, each a whole converged warp.  Warp 1: S = Q K^T into
    //      buffer it % 2 once the PV MMA of tile it - 2 has read P there; warp
    //      3: O (+)= (P_hi + P_lo) V
    constexpr uint32_t idesc_qk = umma_idesc(0, kPfKeys), idesc_pv = umma_idesc(1, kHeadDim);
    uint32_t last_bar = 0;
    int last_par = 0, piece = 0;
    bool ok = true;
    while (ok && walk.next(p, u)) {
      if (warp == 1) {
        ok = __all_sync(kAll, mbar_wait(b_q, piece & 1, abort_flag, p.err));
        tc_fence_after();
      }
      const int n = u.t1 - u.t0;
      for (int j = 0; j < n && ok; ++j, ++it) {
        const int st = it % kTrStages, ph = (it / kTrStages) & 1, buf = it & 1;
        if (warp == 1) {
          ok = __all_sync(kAll, mbar_wait(b_k_full + 8 * st, ph, abort_flag, p.err));
          if (ok && it >= 2)
            ok = __all_sync(kAll,
                            mbar_wait(b_o + 8 * buf, ((it - 2) >> 1) & 1, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t koff = (ks >> 2) * kTrHalf + (ks & 3) * 32;
            const uint32_t qoff = (ks >> 2) * kTrQHalf + (ks & 3) * 32;
            umma_f16_ss(tmem + buf * kTrSCols, umma_desc(base + kTrOffQ + qoff, 16, 1024),
                        umma_desc(base + kTrOffK + st * kTrTile + koff, 16, 1024), idesc_qk,
                        ks > 0);
          }
          umma_commit(b_s + 8 * buf);
          umma_commit(b_k_empty + 8 * st);
          last_bar = b_s + 8 * buf;
        } else {
          ok = __all_sync(kAll, mbar_wait(b_p + 8 * buf, (it >> 1) & 1, abort_flag, p.err));
          if (ok) ok = __all_sync(kAll, mbar_wait(b_v_full + 8 * st, ph, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
          const uint32_t vb = base + kTrOffV + st * kTrTile;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < kPfKeys / 16; ++ks)
              umma_f16_ta(tmem_o, tmem + buf * kTrSCols + part * (kTrSCols / 2) + ks * 8,
                          umma_desc(vb + ks * 16 * 128, kTrHalf, 1024), idesc_pv,
                          (j > 0 || part > 0 || ks > 0) ? 1u : 0u);
          umma_commit(b_o + 8 * buf);
          umma_commit(b_v_empty + 8 * st);
          last_bar = b_o + 8 * buf;
        }
        last_par = (it >> 1) & 1;
      }
      ++piece;
    }
    if (__any_sync(kAll, *abort_flag != 0) && last_bar) {
      // issued MMAs finish before the tensor memory is released
      volatile int never = 0;
      mbar_wait(last_bar, last_par, &never, nullptr);
    }
    __syncwarp();
  } else {
    // ---- softmax warps: TMEM lane quarter warp % 4, a row per thread
    const int lb = 32 * (warp & 3), r = lb + lane;
    const uint32_t trow = (uint32_t)lb << 16;
    const float c = p.scale_log2;
    bool ok = true;
    int piece = 0;
    while (ok && walk.next(p, u)) {
      const int R = u.mt * kPfRows + r;
      const bool valid = R < u.q.nodes * p.group;
      const bool alive = u.mt * kPfRows + lb < u.q.nodes * p.group;  // any row of the warp
      const int node = R / p.group;
      const int done = u.q.keys - u.q.nodes;
      const long long head_row =
          (long long)(u.q.q0 + node) * p.hq + u.g * p.group + R % p.group;
      // Q rows into the layout the TMA gives K tiles
      {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + head_row * kHeadDim);
        uint4 qv[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          qv[i] = valid ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          qv[i].x = (qv[i].x & p.q_and) ^ p.q_xor;
          qv[i].y = (qv[i].y & p.q_and) ^ p.q_xor;
          qv[i].z = (qv[i].z & p.q_and) ^ p.q_xor;
          qv[i].w = (qv[i].w & p.q_and) ^ p.q_xor;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t a = base + kTrOffQ + (i >> 3) * kTrQHalf + sw128(r, i & 7);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(qv[i].x),
                       "r"(qv[i].y), "r"(qv[i].z), "r"(qv[i].w)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(b_q);
      }
      // m: the reference of this row's exponentials (base 2); it moves only when
      // a tile's largest exceeds it by more than 8, so P <= 256 and O is rescaled
      // rarely.  l: the row's sum.  up: the next node of the walk to the root.
      float m = -INFINITY, l = 0.f;
      int up = valid ? node : -1;
      const int32_t *par = p.parents + u.q.q0;
      for (int j = u.t1 - 1; j >= u.t0 && ok; --j, ++it) {
        const int st = it % kTrStages, buf = it & 1;
        const int key0 = j * kPfKeys;
        const bool in_tree = key0 > done - kPfKeys;  // the tile holds drafted nodes
        uint32_t vis[2] = {0u, 0u};
        if (in_tree) {
          if (valid && key0 < done) {
            const int below = done - key0;  // 1 .. 63 committed keys
            vis[0] = below >= 32 ? 0xffffffffu : (1u << below) - 1u;
            vis[1] = below > 32 ? (1u << (below - 32)) - 1u : 0u;
          }
          while (up >= 0 && done + up >= key0) {
            const int k = done + up - key0;
            if (k < 32)
              vis[0] |= 1u << k;
            else if (k < 64)
              vis[1] |= 1u << (k - 32);
            const int next = par[up];
            if (next >= up || next < -1) {
              report(p.err, PA_DEVERR_SHAPE);
              up = -1;
            } else {
              up = next;
            }
          }
        }
        ok = __all_sync(kAll, mbar_wait(b_s + 8 * buf, (it >> 1) & 1, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sb = tmem + buf * kTrSCols;
        if (alive) {
          float sv[2][32];
          tmem_ld64(sb + trow, sv);
          if (in_tree) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                sv[cc][i] = (vis[cc] >> i) & 1u ? sv[cc][i] : -INFINITY;
          }
          float mx8[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) mx8[x] = -INFINITY;
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx8[(i >> 1) & 7] = fmax3(mx8[(i >> 1) & 7], sv[cc][i], sv[cc][i + 1]);
          const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                 fmaxf(mx8[6], mx8[7]));
          const float mxc = mx * c;
          const bool grow = mxc > m + 8.f;
          const float m_new = grow ? mxc : m;
          const float alpha = grow && m != -INFINITY ? exp2f(m - m_new) : 1.f;
          m = m_new;
          const float neg_m = m == -INFINITY ? 0.f : -m;
          const uint64_t c2 = pack_f32x2(c, c), nm2 = pack_f32x2(neg_m, neg_m);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float x0, x1;
              unpack_f32x2(fma_f32x2(pack_f32x2(sv[cc][i], sv[cc][i + 1]), c2, nm2), x0, x1);
              sv[cc][i] = ex2_approx(x0);
              sv[cc][i + 1] = ex2_approx(x1);
            }
          // rows whose reference moved rescale O between the PV of the tile
          // before and this one's
          if (__any_sync(kAll, alpha != 1.f)) {
            ok = __all_sync(kAll, mbar_wait(b_o + 8 * ((it - 1) & 1), ((it - 1) >> 1) & 1,
                                            abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < kHeadDim / 32; ++cc) {
              float ov[32];
              tmem_ld32(tmem_o + trow + cc * 32, ov);
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] *= alpha;
              tmem_st32(tmem_o + trow + cc * 32, ov);
            }
          }
          // P over the scores: hi parts (two keys a column) in the buffer's
          // columns 0 .. 31, lo parts in 32 .. 63
          uint64_t ps4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float e0 = sv[cc >> 1][16 * (cc & 1) + 2 * i];
              const float e1 = sv[cc >> 1][16 * (cc & 1) + 2 * i + 1];
              const uint32_t u0 = __float_as_uint(e0), u1 = __float_as_uint(e1);
              hi[i] = __byte_perm(u0, u1, 0x7632);
              const uint64_t e2 = pack_f32x2(e0, e1);
              ps4[i & 3] = add_f32x2(ps4[i & 3], e2);
              float d0, d1;
              unpack_f32x2(sub_f32x2(e2, pack_f32x2(__uint_as_float(u0 & 0xFFFF0000u),
                                                    __uint_as_float(u1 & 0xFFFF0000u))),
                           d0, d1);
              lo[i] = float2_to_bf16x2(d0, d1);
            }
            tmem_st8(sb + trow + cc * 8, hi);
            tmem_st8(sb + trow + kTrSCols / 2 + cc * 8, lo);
          }
          float ps8[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) unpack_f32x2(ps4[x], ps8[2 * x], ps8[2 * x + 1]);
          l = l * alpha + (((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) +
                           ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7])));
          tmem_wait_st();
        }
        // V rows of the tile that some rows may not see: those past the end may
        // hold anything and are cleared; a drafted node's infinities and NaN are
        // cleared here and put into the rows that see it at the end
        if (in_tree) {
          ok = __all_sync(kAll, mbar_wait(b_v_full + 8 * st, (it / kTrStages) & 1, abort_flag,
                                          p.err));
          if (!ok) break;
          const uint32_t vb = base + kTrOffV + st * kTrTile;
          for (int i = r; i < kPfKeys * 16; i += kPfRows) {
            const int key = key0 + (i >> 4), ch = i & 15;
            if (key < done) continue;
            const uint32_t a = vb + (ch >> 3) * kTrHalf + sw128(i >> 4, ch & 7);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (key < u.q.keys) {
              v = lds128(a);
              const uint4 was = v;
              uint32_t *w = &v.x;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u;
                if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0xffffu;
              }
              if (v.x == was.x && v.y == was.y && v.z == was.z && v.w == was.w) continue;
              *bad_piece = piece;
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x),
                         "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        mbar_arrive(b_p + 8 * buf);
      }
      if (ok)
        ok = __all_sync(kAll, mbar_wait(b_o + 8 * ((it - 1) & 1), ((it - 1) >> 1) & 1, abort_flag,
                                        p.err));
      if (!ok) break;
      tc_fence_after();
      if (alive) {
        const bool bad = *bad_piece == piece;
        const bool whole = u.t0 == 0 && u.t1 == u.tiles;
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (l NaN: a NaN row)
        const long long slot = ((u.t0 > 0 ? 0 : (long long)p.splits) + blockIdx.x) * kPfRows + r;
        float *dst32 = whole ? static_cast<float *>(p.out) + head_row * kHeadDim
                             : p.part_o + slot * kHeadDim;
        uint16_t *dst16 = static_cast<uint16_t *>(p.out) + head_row * kHeadDim;
#pragma unroll 1
        for (int cc = 0; cc < kHeadDim / 32; ++cc) {
          float ov[32];
          tmem_ld32(tmem_o + trow + cc * 32, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] *= inv;
          if (valid) {
            if (bad) {
              const uint32_t dims = not_finite(p, u.s, u.q.q0, done, u.g, node, u.t0 * kPfKeys,
                                               u.t1 * kPfKeys - 1, cc);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if ((dims >> i) & 1u) ov[i] = __int_as_float(0x7fffffff);
            }
            if (whole && !p.out_f32) {
              uint4 *dst = reinterpret_cast<uint4 *>(dst16 + cc * 32);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_uint4(float2_to_bf16x2(ov[8 * i], ov[8 * i + 1]),
                                    float2_to_bf16x2(ov[8 * i + 2], ov[8 * i + 3]),
                                    float2_to_bf16x2(ov[8 * i + 4], ov[8 * i + 5]),
                                    float2_to_bf16x2(ov[8 * i + 6], ov[8 * i + 7]));
            } else {
              float4 *dst = reinterpret_cast<float4 *>(dst32 + cc * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
            }
          }
          __syncwarp();
        }
        if (valid && !whole)
          p.part_lse[slot] = l == 0.f ? -INFINITY : m + log2f(l);
      }
      tc_fence_before();
      ++piece;
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTrCols)
                 : "memory");
  }
}

// ---- merge --------------------------------------------------------------------
// One CTA per (token, query head): where the token's unit was cut, its row is
// sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M) over the unit's pieces.  Each of
// four warps takes a quarter of them, eight rows of loads in flight, a lane
// four dims.
constexpr int kTmWarps = 4;

__global__ void __launch_bounds__(32 * kTmWarps) tree_merge_kernel(const TreeParams p) {
  __shared__ long long warp_sum[kTmWarps];
  __shared__ long long unit_start;
  __shared__ int unit_seq;
  __shared__ float share_m[kTmWarps], share_w[kTmWarps];
  __shared__ float4 share_o[kTmWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x, h = blockIdx.y, g = h / p.group;
  if (tid == 0) unit_seq = -1;
  const int per = (p.num_seqs + 32 * kTmWarps - 1) / (32 * kTmWarps);
  const int s0 = min(p.num_seqs, tid * per), s1 = min(p.num_seqs, s0 + per);
  long long mine = 0, N;
  for (int s = s0; s < s1; ++s) mine += head_weight(tree_seq(p, s, false), p.group) * p.hkv;
  long long before = block_before(mine, warp_sum, N);
  const long long C = ctas_in_use(p, N);
  for (int s = s0; s < s1; ++s) {
    const TreeSeq q = tree_seq(p, s, false);
    const long long w = head_weight(q, p.group);
    if (q.nodes > 0 && t >= q.q0 && t < q.q0 + q.nodes) {
      unit_seq = s;
      unit_start = before + w * g;
    }
    before += w * p.hkv;
  }
  __syncthreads();
  if (unit_seq < 0) return;  // a row of no sequence
  const TreeSeq q = tree_seq(p, unit_seq, false);
  const int R = (t - q.q0) * p.group + h % p.group, mt = R / kPfRows, r = R % kPfRows;
  long long U = unit_start;
  for (int i = 0; i < mt; ++i) U += unit_tiles(q, p.group, i) + kTrPieceTiles;
  const long long c0 = cta_of(U, C, N), c1 = cta_of(U + unit_tiles(q, p.group, mt) - 1, C, N);
  if (c0 == c1) return;  // in one piece: written already
  const long long len = (c1 - c0 + kTmWarps) / kTmWarps;
  const long long ca = c0 + warp * len, cb = min(c1 + 1, ca + len);
  float M = -INFINITY, W = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;
  for (long long x = ca; x < cb; x += kBatch) {
    float lse[kBatch];
    float4 o[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      lse[i] = -INFINITY;
      o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x + i < cb) {
        const long long slot = ((x + i == c0 ? (long long)p.splits : 0) + x + i) * kPfRows + r;
        lse[i] = p.part_lse[slot];
        o[i] = reinterpret_cast<const float4 *>(p.part_o + slot * kHeadDim)[lane];
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, lse[i]);
    const float ref = top == -INFINITY ? 0.f : top;  // nothing seen so far: weights zero
    const float old = exp2f(M - ref);
    W *= old;
    acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = exp2f(lse[i] - ref);
      if (w == 0.f) continue;
      W += w;
      acc.x = fmaf(w, o[i].x, acc.x);
      acc.y = fmaf(w, o[i].y, acc.y);
      acc.z = fmaf(w, o[i].z, acc.z);
      acc.w = fmaf(w, o[i].w, acc.w);
    }
    M = top;
  }
  share_o[warp][lane] = acc;
  if (lane == 0) {
    share_m[warp] = M;
    share_w[warp] = W;
  }
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < kTmWarps; ++w)
    if (!(share_w[w] == 0.f)) top = fmaxf(top, share_m[w]);
  float sum = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kTmWarps; ++w) {
    if (share_w[w] == 0.f) continue;
    const float f = exp2f(share_m[w] - top);
    const float4 a = share_o[w][lane];
    sum = fmaf(f, share_w[w], sum);
    acc.x = fmaf(f, a.x, acc.x);
    acc.y = fmaf(f, a.y, acc.y);
    acc.z = fmaf(f, a.z, acc.z);
    acc.w = fmaf(f, a.w, acc.w);
  }
  const float inv = sum > 0.f ? 1.f / sum : sum;
  acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
  const long long row = ((long long)t * p.hq + h) * kHeadDim + lane * 4;
  if (p.out_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row) = acc;
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row) =
        make_uint2(float2_to_bf16x2(acc.x, acc.y), float2_to_bf16x2(acc.z, acc.w));
}

constexpr size_t kTrHead = 256;  // the error word
size_t tree_part_bytes(long long splits) {
  return (size_t)splits * 2 * kPfRows * kHeadDim * sizeof(float);
}
size_t tree_workspace(long long splits) {
  return kTrHead + tree_part_bytes(splits) + (size_t)splits * 2 * kPfRows * sizeof(float);
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_tree_workspace_size(int32_t num_splits) {
  if (num_splits < 1 || num_splits > PA_DECODE_MAX_SPLITS) return 0;
  return pa::tree_workspace(num_splits);
}

extern "C" int32_t pa_decode_tree_default_splits(int32_t device) {
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return -1;
  return 2 * sms;
}

extern "C" pa_status pa_decode_tree(void *out, int32_t out_dtype, const void *q,
                                    const int32_t *cu_seqlens, const int32_t *parents,
                                    int32_t num_seqs, int32_t total_tokens, int32_t max_q_len,
                                    const void *k_cache, const void *v_cache, int64_t num_blocks,
                                    const int32_t *block_tables, int32_t block_table_stride,
                                    const int32_t *context_lens, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    float scale, int32_t num_splits, void *workspace,
                                    size_t workspace_bytes, uint32_t flags, void *stream) {
  using namespace pa;
  if (num_seqs < 0 || total_tokens < 0 || max_q_len < 0 || num_blocks < 0 || num_splits < 0 ||
      num_splits > PA_DECODE_MAX_SPLITS)
    return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (out_dtype != PA_DTYPE_BF16 && out_dtype != PA_DTYPE_F32) return PA_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (!(num_kv_heads == 1 || num_kv_heads == 2 || num_kv_heads == 4 || num_kv_heads == 8))
    return PA_ERR_UNSUPPORTED;
  if (num_q_heads < num_kv_heads || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 8)
    return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_tokens == 0 || max_q_len == 0) return PA_OK;
  if (num_blocks < 1 || num_blocks > INT_MAX / kBlockSize || block_table_stride < 1)
    return PA_ERR_INVALID_ARG;
  if (!out || !q || !cu_seqlens || !parents || !k_cache || !v_cache || !block_tables ||
      !context_lens)
    return PA_ERR_INVALID_ARG;
  auto off = [](const void *x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) % a) != 0; };
  if (off(out, 16) || off(q, 16) || off(k_cache, 16) || off(v_cache, 16) || off(workspace, 16) ||
      off(cu_seqlens, 4) || off(parents, 4) || off(block_tables, 4) || off(context_lens, 4))
    return PA_ERR_INVALID_ARG;
  if (!workspace) return PA_ERR_WORKSPACE;
  if (num_splits > 0 && workspace_bytes < tree_workspace(num_splits)) return PA_ERR_WORKSPACE;
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_DEVICE;
  const int splits = num_splits > 0 ? num_splits : pa_decode_tree_default_splits(device);
  if (splits < 1) return PA_ERR_DEVICE;
  if (workspace_bytes < tree_workspace(splits)) return PA_ERR_WORKSPACE;
  CUtensorMap tk, tv;
  memset(&tk, 0, sizeof tk);
  memset(&tv, 0, sizeof tv);
  if (!pf_pool_map(&tk, k_cache, num_blocks, num_kv_heads) ||
      !pf_pool_map(&tv, v_cache, num_blocks, num_kv_heads))
    return PA_ERR_DEVICE;
  static std::atomic<bool> configured[64] = {};
  if (set_smem_once(configured, tree_kernel, device, kTrSmem) != cudaSuccess) return PA_ERR_LAUNCH;
  // two CTAs per SM: all of the unified L1 / shared memory as shared memory (a hint)
  cudaFuncSetAttribute(tree_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  char *ws = static_cast<char *>(workspace);
  TreeParams p;
  p.out = out;
  p.out_f32 = out_dtype == PA_DTYPE_F32;
  p.q = static_cast<const uint16_t *>(q);
  p.cu = cu_seqlens;
  p.parents = parents;
  p.num_seqs = num_seqs;
  p.total_tokens = total_tokens;
  p.max_q_len = max_q_len;
  p.v_cache = static_cast<const uint16_t *>(v_cache);
  p.num_blocks = num_blocks;
  p.tables = block_tables;
  p.bt_stride = block_table_stride;
  p.ctx = context_lens;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  // masked scores are -inf before scaling, which needs a positive factor: a
  // negative scale flips q's signs, a zero one makes q zero
  p.scale_log2 = (scale > 0.f ? scale : scale < 0.f ? -scale : 1.f) * 1.4426950408889634f;
  p.q_and = scale == 0.f ? 0u : 0xFFFFFFFFu;
  p.q_xor = scale < 0.f ? 0x80008000u : 0u;
  p.splits = splits;
  p.all_splits = num_splits > 0;
  p.part_o = reinterpret_cast<float *>(ws + kTrHead);
  p.part_lse = reinterpret_cast<float *>(ws + kTrHead + tree_part_bytes(splits));
  p.err = static_cast<int32_t *>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_kernel(tree_kernel, dim3((unsigned)splits), dim3(kTrThreads), kTrSmem, s, true, tk,
                    tv, p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  if (splits > 1 &&
      launch_kernel(tree_merge_kernel, dim3((unsigned)total_tokens, (unsigned)num_q_heads),
                    dim3(32 * kTmWarps), 0, s, true, p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}
