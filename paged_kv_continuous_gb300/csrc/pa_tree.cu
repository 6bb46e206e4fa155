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
// K is needed a step before V of the same tile, and a loaded memory system takes
// longer than a step: three K stages and two V stages, all the shared memory that
// leaves room for two CTAs on an SM (so nothing is declared static).
#ifndef TR_KST
#define TR_KST 3
#endif
constexpr int kTrKStages = TR_KST, kTrVStages = 2;
constexpr int kTrOffQ = 0;
constexpr int kTrOffK = kTrOffQ + 2 * kTrQHalf;
constexpr int kTrOffV = kTrOffK + kTrKStages * kTrTile;
constexpr int kTrOffBar = kTrOffV + kTrVStages * kTrTile;
// 8-byte slots: K full / empty and V full / empty per stage, Q, two score, two
// P and two PV barriers, the TMEM address, the abort flag, the last piece with
// a V row that is not finite, the sums of the plan's scan, the CTA's place
constexpr int kTsKFull = 0, kTsKEmpty = kTsKFull + kTrKStages, kTsVFull = kTsKEmpty + kTrKStages;
constexpr int kTsVEmpty = kTsVFull + kTrVStages, kTsQ = kTsVEmpty + kTrVStages, kTsS = kTsQ + 1;
constexpr int kTsP = kTsS + 2, kTsO = kTsP + 2, kTsTmem = kTsO + 2, kTsAbort = kTsTmem + 1;
constexpr int kTsBad = kTsAbort + 1, kTsSum = kTsBad + 1, kTsPlace = kTsSum + kTrThreads / 32;
constexpr int kTsSlots = 48;
constexpr int kTrSmem = kTrOffBar + kTsSlots * 8;
static_assert(2 * (kTrSmem + 1024) <= 228 * 1024, "two CTAs do not fit an SM");
constexpr int kTrCols = 256;    // tensor memory columns: S_0 0.., S_1 64.., O 128..
constexpr int kTrSCols = 64, kTrO = 128;

#ifndef TR_PIECE
#define TR_PIECE 2
#endif
#ifndef TR_MIN
#define TR_MIN 4
#endif
// A piece's start and end cost about as much as this many tiles.
constexpr int kTrPieceTiles = TR_PIECE;
// A CTA's part of the list is at least this long.
constexpr int kTrMinPart = TR_MIN;

// What the merge has to know of CTA c's first piece, where it goes on with a unit
// that an earlier CTA began: the unit's rows, CTAs first .. last and output rows.
struct TreeCut {
  int rows, first, last;  // rows 0: the CTA starts with a unit's first tile
  int q0, g, mt, unused[2];
};

#ifndef TR_X
#define TR_X
#endif
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
  uint32_t group_inv;     // ceil(2^32 / group): x / group = umulhi(x, group_inv) (x < 2^29)
  float scale_log2;       // > 0: a scale <= 0 is folded into q as staged
  uint32_t q_and, q_xor;  // staged q pairs = (q & q_and) ^ q_xor
  int splits;             // CTAs of the launch
  int min_part;
  TreeCut *cuts;          // [splits]
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

__device__ __forceinline__ int by_group(const TreeParams &p, int x) {
  return p.group == 1 ? x : (int)__umulhi((uint32_t)x, p.group_inv);
}
// Tiles of row tile mt: up to the key of its last node.
__device__ __forceinline__ int unit_tiles(const TreeParams &p, const TreeSeq &q, int mt) {
  const int last = by_group(p, min((mt + 1) * kPfRows, q.nodes * p.group) - 1);
  return (int)((unsigned)(q.keys - q.nodes + last) / kPfKeys) + 1;
}
__device__ __forceinline__ int row_tiles(const TreeParams &p, const TreeSeq &q) {
  return (int)((unsigned)(q.nodes * p.group + kPfRows - 1) / kPfRows);
}
// Length of one kv head of the sequence in the list.
__device__ __forceinline__ long long head_weight(const TreeParams &p, const TreeSeq &q) {
  long long w = 0;
  const int m = row_tiles(p, q);
  for (int i = 0; i < m; ++i) w += unit_tiles(p, q, i) + kTrPieceTiles;
  return w;
}

// The list is cut into parts of this length, one for a CTA, while it lasts.
__device__ __forceinline__ long long part_length(const TreeParams &p, long long N) {
  const long long len = N < (1ll << 31) ? ((unsigned)N + (unsigned)p.splits - 1u) / (unsigned)p.splits
                                        : (N + p.splits - 1) / p.splits;
  return max((long long)p.min_part, len);
}
__device__ __forceinline__ int part_of(long long x, long long len) {
  return x < (1ll << 31) && len < (1ll << 31) ? (int)((unsigned)x / (unsigned)len) : (int)(x / len);
}

// What lies before this thread's share of the list, and the whole.
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
#pragma unroll
  for (int w = 0; w < kTrThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  return before;
}

// A CTA's place in the list: the unit it is in and where that unit starts.
struct TreePlace {
  long long x, end, start;
  int s, g, mt;
  TreeSeq q;
};
static_assert(sizeof(TreePlace) <= (kTsSlots - kTsPlace) * 8, "the place does not fit");

struct TreePiece {
  TreeSeq q;
  int s, g, mt, t0, t1, tiles;
};

// The next piece of a CTA's part of the list; every warp runs this for itself.
struct TreeWalk {
  TreePlace at;

  __device__ __forceinline__ bool next(const TreeParams &p, TreePiece &r) {
    while (at.x < at.end) {
      const int tiles = unit_tiles(p, at.q, at.mt);
      const long long rel = at.x - at.start;
      const bool got = rel < tiles;
      if (got) {
        r.q = at.q;
        r.s = at.s;
        r.g = at.g;
        r.mt = at.mt;
        r.tiles = tiles;
        r.t0 = (int)rel;
        r.t1 = (int)min((long long)tiles, at.end - at.start);
      }
      at.start += tiles + kTrPieceTiles;
      at.x = at.start;
      if (++at.mt == row_tiles(p, at.q)) {
        at.mt = 0;
        if (++at.g == p.hkv) {
          at.g = 0;
          if (at.x < at.end) do {
              at.q = tree_seq(p, ++at.s, false);
            } while (at.q.nodes == 0 && at.s + 1 < p.num_seqs);
        }
      }
      if (got) return true;
    }
    return false;
  }
};

// The CTA's part of the list: the thread whose sequences hold its start leaves the
// place there.  False: nothing to do.
__device__ __forceinline__ bool tree_plan(const TreeParams &p, long long *warp_sum,
                                          TreePlace *place, long long &len) {
  const int per = (int)((unsigned)p.num_seqs + kTrThreads - 1u) / kTrThreads;
  const int s0 = min(p.num_seqs, (int)threadIdx.x * per), s1 = min(p.num_seqs, s0 + per);
  long long mine = 0, N;
  TreeSeq q = {0, 0, 0};
  for (int s = s0; s < s1; ++s) {
    q = tree_seq(p, s, blockIdx.x == 0);
    mine += head_weight(p, q) * p.hkv;
  }
  long long before = block_before(mine, warp_sum, N);
  len = part_length(p, N);
  const long long x0 = (long long)blockIdx.x * len;
  if (x0 >= N) return false;
  if (x0 < before || x0 >= before + mine) return true;
  for (int s = s0; s < s1; ++s) {
    if (per > 1) q = tree_seq(p, s, false);
    const long long w = head_weight(p, q);
    if (x0 < before + w * p.hkv) {
      TreePlace r;
      r.x = x0;
      r.end = min(N, x0 + len);
      r.s = s;
      r.q = q;
      r.g = 0;
      r.start = before;
      while (x0 >= r.start + w) {
        r.start += w;
        ++r.g;
      }
      r.mt = 0;
      while (true) {
        const int unit = unit_tiles(p, q, r.mt) + kTrPieceTiles;
        if (x0 < r.start + unit) break;
        r.start += unit;
        ++r.mt;
      }
      *place = r;
      break;
    }
    before += w * p.hkv;
  }
  return true;
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
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_addr(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kTrOffBar);
  const uint32_t b_k_full = smem_addr(bars + kTsKFull), b_k_empty = smem_addr(bars + kTsKEmpty);
  const uint32_t b_v_full = smem_addr(bars + kTsVFull), b_v_empty = smem_addr(bars + kTsVEmpty);
  const uint32_t b_q = smem_addr(bars + kTsQ), b_s = smem_addr(bars + kTsS);
  const uint32_t b_p = smem_addr(bars + kTsP), b_o = smem_addr(bars + kTsO);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kTsTmem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kTsAbort);
  volatile int *bad_piece = reinterpret_cast<volatile int *>(bars + kTsBad);
  long long *warp_sum = reinterpret_cast<long long *>(bars + kTsSum);
  TreePlace *place = reinterpret_cast<TreePlace *>(bars + kTsPlace);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < kTrKStages; ++i) {
      mbar_init(b_k_full + 8 * i, 1);
      mbar_init(b_k_empty + 8 * i, 1);
    }
    for (int i = 0; i < kTrVStages; ++i) {
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
  if (warp == 1) {
    // (another kernel's CTAs on this SM may hold it: this waits until they end)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTrCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  griddep_wait();
  griddep_launch_dependents();
  long long len;
  const bool busy = tree_plan(p, warp_sum, place, len) && (base & 1023) == 0;
  // (the swizzle needs it; without static shared memory the base is aligned)
  if ((base & 1023) != 0 && tid == 0) report(p.err, PA_DEVERR_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + kTrO;
  TreeWalk walk;
  if (busy)
    walk.at = *place;
  else
    walk.at.x = walk.at.end = walk.at.start = 0;
  if (tid == 96) {
    TreeCut cut = {};
    const long long rel = walk.at.x - walk.at.start;
    const int tiles = busy ? unit_tiles(p, walk.at.q, walk.at.mt) : 0;
    if (busy && rel > 0 && rel < tiles) {
      cut.rows = min(kPfRows, walk.at.q.nodes * p.group - walk.at.mt * kPfRows);
      cut.first = part_of(walk.at.start, len);
      cut.last = part_of(walk.at.start + tiles - 1, len);
      cut.q0 = walk.at.q.q0;
      cut.g = walk.at.g;
      cut.mt = walk.at.mt;
    }
    p.cuts[blockIdx.x] = cut;
  }
  __syncwarp();
  constexpr unsigned kAll = 0xffffffffu;

  TreePiece u;
  int it = 0;  // tiles done so far, over all pieces; tile it's scores are in buffer it % 2

  if (warp == 0 || warp == 2) {
    // ---- loaders: a tile's pages (64 dims x 16 keys a box) into the next stage
    //      once the MMAs that read its previous tile are done
    const bool is_k = warp == 0;
    const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
    const uint32_t dst0 = base + (is_k ? kTrOffK : kTrOffV);
    const uint32_t full0 = is_k ? b_k_full : b_v_full, empty0 = is_k ? b_k_empty : b_v_empty;
    const int stages = is_k ? kTrKStages : kTrVStages;
    constexpr int kChunk = 32 / kTrPages;  // tiles whose table entries a warp holds
    int st = 0, par = 0;                   // stage, and the parity of its round
    bool ok = true;
    while (ok && walk.next(p, u)) {
      const int32_t *row = p.tables + (long long)u.s * p.bt_stride;
      // an entry per lane, and those of the next eight tiles on their way: -1 no
      // key in the page (left as it is: masked), -2 a bad entry
      auto entry = [&](int chunk) {
        const long long page = (long long)chunk * 32 + lane;
        const bool has = chunk >= 0 && page * kBlockSize < u.q.keys;
        const int ph = has ? row[page] : -1;
        return !has ? -1 : ph >= 0 && ph < p.num_blocks ? ph : -2;
      };
      int chunk = (u.t1 - 1) / kChunk;
      int ph_lane = entry(chunk), ph_next = entry(chunk - 1);
      for (int j = u.t1 - 1; j >= u.t0; --j, ++it) {
        if (j / kChunk != chunk) {
          --chunk;
          ph_lane = ph_next;
          ph_next = entry(chunk - 1);
        }
        if (it >= stages &&
            !__all_sync(kAll, mbar_wait(empty0 + 8 * st, par ^ 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        const int at = (j % kChunk) * kTrPages;
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
        if (++st == stages) st = 0, par ^= 1;
      }
    }
    if (lane == 0 && *abort_flag) {
      // copies in flight must land before the CTA's shared memory is released
      volatile int never = 0;
      for (int i = it > stages ? it - stages : 0; i < it; ++i)
        mbar_wait(full0 + 8 * (i % stages), (i / stages) & 1, &never, nullptr);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers, each a whole converged warp.  Warp 1: S = Q K^T into
    //      buffer it % 2 once the PV MMA of tile it - 2 has read P there; warp
    //      3: O (+)= (P_hi + P_lo) V
    constexpr uint32_t idesc_qk = umma_idesc(0, kPfKeys), idesc_pv = umma_idesc(1, kHeadDim);
    uint32_t last_bar = 0;
    int last_par = 0, piece = 0, st = 0, ph = 0;  // (of this warp's operand)
    bool ok = true;
    while (ok && walk.next(p, u)) {
      if (warp == 1) {
        ok = __all_sync(kAll, mbar_wait(b_q, piece & 1, abort_flag, p.err));
        tc_fence_after();
      }
      const int n = u.t1 - u.t0;
      for (int j = 0; j < n && ok; ++j, ++it) {
        const int buf = it & 1;
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
          if (++st == kTrKStages) st = 0, ph ^= 1;
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
          if (++st == kTrVStages) st = 0, ph ^= 1;
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
      const int R = u.mt * kPfRows + r, limit = u.q.nodes * p.group;
      const bool valid = R < limit;
      const bool alive = u.mt * kPfRows + lb < limit;  // any row of the warp
      const int node = by_group(p, R);
      const int done = u.q.keys - u.q.nodes;
      // row R of the tile is this row of q and out
      auto head_row = [&](int x) {
        const int n = by_group(p, x);
        return (long long)(u.q.q0 + n) * p.hq + u.g * p.group + (x - n * p.group);
      };
      // Q rows, half a warp a row, into the layout the TMA gives K tiles
      if (alive) {
        uint4 qv[16];
        const int ch = lane & 15;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = u.mt * kPfRows + lb + 2 * i + (lane >> 4);
          qv[i] = make_uint4(0u, 0u, 0u, 0u);
          if (x < limit) qv[i] = reinterpret_cast<const uint4 *>(p.q + head_row(x) * kHeadDim)[ch];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t a = base + kTrOffQ + (ch >> 3) * kTrQHalf +
                             sw128(lb + 2 * i + (lane >> 4), ch & 7);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a),
                       "r"((qv[i].x & p.q_and) ^ p.q_xor), "r"((qv[i].y & p.q_and) ^ p.q_xor),
                       "r"((qv[i].z & p.q_and) ^ p.q_xor), "r"((qv[i].w & p.q_and) ^ p.q_xor)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      mbar_arrive(b_q);
      // m: the reference of this row's exponentials (base 2); it moves only when
      // a tile's largest exceeds it by more than 8, so P <= 256 and O is rescaled
      // rarely.  l: the row's sum.  up: the next node of the walk to the root.
      float m = -INFINITY, l = 0.f;
      // A tile's 64 keys are a window of 64 nodes, whose parents the warp holds,
      // two a lane: a step of the walk is a shuffle.
      int up = valid ? node : -1;
      const int32_t *par = p.parents + u.q.q0;
      auto climb = [&](int first, uint32_t (&vis)[2]) {  // window first .. first + 63
        const int n0 = first + lane, n1 = n0 + 32;
        const int par0 = n0 >= 0 && n0 < u.q.nodes ? par[n0] : -1;
        const int par1 = n1 >= 0 && n1 < u.q.nodes ? par[n1] : -1;
        while (__any_sync(kAll, up >= 0 && up >= first)) {
          const int k = up - first;
          const int next0 = __shfl_sync(kAll, par0, k & 31), next1 = __shfl_sync(kAll, par1, k & 31);
          if (up < 0 || k < 0) continue;
          if (k < 32)
            vis[0] |= 1u << k;
          else
            vis[1] |= 1u << (k - 32);
          const int next = k < 32 ? next0 : next1;
          if (next >= up || next < -1) report(p.err, PA_DEVERR_SHAPE);
          up = next < up && next >= -1 ? next : -1;
        }
      };
      if (alive && u.t1 * kPfKeys > done) {  // the windows above the piece's last tile
        uint32_t unused[2] = {0u, 0u};
        const int top = by_group(p, min(u.mt * kPfRows + lb + 31, limit - 1));
        for (int j = (done + top) / kPfKeys; j >= u.t1; --j) climb(j * kPfKeys - done, unused);
      }
      for (int j = u.t1 - 1; j >= u.t0 && ok; --j, ++it) {
        const int st = it % kTrVStages, buf = it & 1;
        const int key0 = j * kPfKeys;
        const bool in_tree = key0 > done - kPfKeys;  // the tile holds drafted nodes
        uint32_t vis[2] = {0u, 0u};
        if (in_tree && alive) {
          climb(key0 - done, vis);
          if (valid && key0 < done) {
            const int below = done - key0;  // 1 .. 63 committed keys
            vis[0] |= below >= 32 ? 0xffffffffu : (1u << below) - 1u;
            vis[1] |= below > 32 ? (1u << (below - 32)) - 1u : 0u;
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
          ok = __all_sync(kAll, mbar_wait(b_v_full + 8 * st, (it / kTrVStages) & 1, abort_flag,
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
        const long long slot = ((u.t0 > 0 ? 0 : (long long)p.splits) + blockIdx.x) * kPfRows + lb;
        // 32 columns of the warp's rows at a time go through its own Q rows (which
        // no MMA reads any more), so that eight lanes store a row's 128 bytes
        const uint32_t stage = base + kTrOffQ + lb * 128;
        const int x0 = lane >> 3, col = 4 * (lane & 7);
        char *dst[8];  // of rows x0 + 4 i; null: no such row
        const bool narrow = whole && !p.out_f32;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int x = u.mt * kPfRows + lb + x0 + 4 * i;
          const long long at = whole ? head_row(x) : slot + x0 + 4 * i;
          dst[i] = static_cast<char *>(whole ? p.out : static_cast<void *>(p.part_o)) +
                   (at * kHeadDim + col) * (narrow ? 2 : 4);
          if (x >= limit) dst[i] = nullptr;
        }
#pragma unroll 1
        for (int cc = 0; cc < kHeadDim / 32; ++cc) {
          float ov[32];
          tmem_ld32(tmem_o + trow + cc * 32, ov);
          if (valid && bad TR_X) {
            const uint32_t dims = not_finite(p, u.s, u.q.q0, done, u.g, node, u.t0 * kPfKeys,
                                             u.t1 * kPfKeys - 1, cc);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((dims >> i) & 1u) ov[i] = __int_as_float(0x7fffffff);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + sw128(lane, i)),
                         "f"(ov[4 * i] * inv), "f"(ov[4 * i + 1] * inv), "f"(ov[4 * i + 2] * inv),
                         "f"(ov[4 * i + 3] * inv)
                         : "memory");
          __syncwarp();
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = lds128(stage + sw128(x0 + 4 * i, lane & 7));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (dst[i] == nullptr) continue;
            if (narrow)
              *reinterpret_cast<uint2 *>(dst[i] + cc * 64) =
                  make_uint2(float2_to_bf16x2(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                             float2_to_bf16x2(__uint_as_float(w[i].z), __uint_as_float(w[i].w)));
            else
              *reinterpret_cast<uint4 *>(dst[i] + cc * 128) = w[i];
          }
        }
        __syncwarp();
        if (valid && !whole)
          p.part_lse[slot + lane] = l == 0.f ? -INFINITY : m + log2f(l);
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
// Row r of a cut unit is sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M) over its
// pieces, M the largest lse.  CTA c serves the unit that part c went on with:
// such a unit of n + 1 pieces has n of these CTAs, and the i-th of them takes
// rows i, i + n, ..., so every CTA reads about one piece's worth of rows however
// long the unit is.  A row is one warp's, or several warps' that share its pieces
// where a CTA has few rows; eight loads of 512 bytes in flight each.
constexpr int kTmWarps = 8;

struct RowSum {
  float m, w;
  float4 o;
};
__device__ __forceinline__ void row_add(RowSum &a, float w, const float4 &o) {
  a.w += w;
  a.o.x = fmaf(w, o.x, a.o.x);
  a.o.y = fmaf(w, o.y, a.o.y);
  a.o.z = fmaf(w, o.z, a.o.z);
  a.o.w = fmaf(w, o.w, a.o.w);
}

__global__ void __launch_bounds__(32 * kTmWarps) tree_merge_kernel(const TreeParams p) {
  __shared__ float share_m[kTmWarps], share_w[kTmWarps];
  __shared__ float4 share_o[kTmWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TreeCut cut = p.cuts[blockIdx.x];
  if (cut.rows == 0) return;
  const int n = cut.last - cut.first, i0 = (int)blockIdx.x - cut.first - 1;
  const int rows = (cut.rows - i0 + n - 1) / n;  // rows of this CTA
  // warps that share a row
  const int share = rows >= 5 ? 1 : rows >= 3 ? 2 : rows == 2 ? 4 : 8;
  const int each = (n + share) / share;  // pieces of a warp
  const int ca = cut.first + (warp % share) * each, cb = min(cut.last + 1, ca + each);
  for (int k = 0; k < rows; k += kTmWarps / share) {
    const int r = i0 + (k + warp / share) * n;
    const bool mine = r < cut.rows;
    RowSum a = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    constexpr int kBatch = 8;
    for (int x = ca; mine && x < cb; x += kBatch) {
      float lse[kBatch];
      float4 o[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        lse[i] = -INFINITY;
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x + i < cb) {
          const long long slot =
              ((x + i == cut.first ? (long long)p.splits : 0) + x + i) * kPfRows + r;
          lse[i] = p.part_lse[slot];
          o[i] = reinterpret_cast<const float4 *>(p.part_o + slot * kHeadDim)[lane];
        }
      }
      float top = a.m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) top = fmaxf(top, lse[i]);
      const float ref = top == -INFINITY ? 0.f : top;  // nothing seen so far: weights zero
      const float old = exp2f(a.m - ref);
      a.w *= old;
      a.o.x *= old, a.o.y *= old, a.o.z *= old, a.o.w *= old;
      a.m = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float w = exp2f(lse[i] - ref);
        if (!(w == 0.f)) row_add(a, w, o[i]);
      }
    }
    if (share > 1) {
      share_o[warp][lane] = a.o;
      if (lane == 0) {
        share_m[warp] = a.m;
        share_w[warp] = a.w;
      }
      __syncthreads();
      if (warp % share == 0) {
        float top = -INFINITY;
        for (int w = warp; w < warp + share; ++w)
          if (!(share_w[w] == 0.f)) top = fmaxf(top, share_m[w]);
        a = {top, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int w = warp; w < warp + share; ++w) {
          if (share_w[w] == 0.f) continue;
          const float f = exp2f(share_m[w] - top);
          const float4 o = share_o[w][lane];
          a.w = fmaf(f, share_w[w], a.w);
          a.o.x = fmaf(f, o.x, a.o.x);
          a.o.y = fmaf(f, o.y, a.o.y);
          a.o.z = fmaf(f, o.z, a.o.z);
          a.o.w = fmaf(f, o.w, a.o.w);
        }
      }
      __syncthreads();
    }
    if (!mine || warp % share != 0) continue;
    const float inv = a.w > 0.f ? 1.f / a.w : a.w;
    const int R = cut.mt * kPfRows + r, node = by_group(p, R);
    const long long at = ((long long)(cut.q0 + node) * p.hq + cut.g * p.group +
                          (R - node * p.group)) * kHeadDim + lane * 4;
    const float4 o = make_float4(a.o.x * inv, a.o.y * inv, a.o.z * inv, a.o.w * inv);
    if (p.out_f32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = o;
    else
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
          make_uint2(float2_to_bf16x2(o.x, o.y), float2_to_bf16x2(o.z, o.w));
  }
}

constexpr size_t kTrHead = 256;  // the error word
size_t tree_part_bytes(long long splits) {
  return (size_t)splits * 2 * kPfRows * kHeadDim * sizeof(float);
}
size_t tree_lse_bytes(long long splits) { return (size_t)splits * 2 * kPfRows * sizeof(float); }
size_t tree_workspace(long long splits) {
  return kTrHead + tree_part_bytes(splits) + tree_lse_bytes(splits) +
         (size_t)splits * sizeof(TreeCut);
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
  if (total_tokens > (1 << 26)) return PA_ERR_UNSUPPORTED;  // (rows of a kv head below 2^29)
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
  p.group_inv = (uint32_t)(((1ull << 32) + p.group - 1) / p.group);
  // masked scores are -inf before scaling, which needs a positive factor: a
  // negative scale flips q's signs, a zero one makes q zero
  p.scale_log2 = (scale > 0.f ? scale : scale < 0.f ? -scale : 1.f) * 1.4426950408889634f;
  p.q_and = scale == 0.f ? 0u : 0xFFFFFFFFu;
  p.q_xor = scale < 0.f ? 0x80008000u : 0u;
  p.splits = splits;
  p.min_part = num_splits > 0 ? 1 : kTrMinPart;
  p.part_o = reinterpret_cast<float *>(ws + kTrHead);
  p.part_lse = reinterpret_cast<float *>(ws + kTrHead + tree_part_bytes(splits));
  p.cuts = reinterpret_cast<TreeCut *>(ws + kTrHead + tree_part_bytes(splits) +
                                       tree_lse_bytes(splits));
  p.err = static_cast<int32_t *>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_kernel(tree_kernel, dim3((unsigned)splits), dim3(kTrThreads), kTrSmem, s, true, tk,
                    tv, p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  if (splits > 1 &&
      launch_kernel(tree_merge_kernel, dim3((unsigned)splits), dim3(32 * kTmWarps), 0, s, true,
                    p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}
