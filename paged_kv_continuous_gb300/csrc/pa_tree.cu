// pa_decode_tree: attention of trees of drafted tokens over the paged bf16
// cache.  Node i of a sequence with P committed keys sees keys 0 .. P - 1 and
// the nodes on its way to the root (keys P + a), so with rows (node, head)
//   S = Q K^T,  P = exp2(c S - m) where seen,  O = P V,  l = sum P,  out = O / l
// and every key is read once for all the nodes and all the G query heads of its
// kv head.
//
// A unit is a 128-row tile of one (sequence, kv head); its keys are cut into
// 64-key tiles.  Units' tiles form lists (sequence, kv head, row tile) that are cut
// evenly over the CTAs, two per SM: a CTA runs the last tiles of one unit, some
// whole units and the first tiles of another.  A unit in one piece is written to
// `out`; the pieces of a cut one leave (O / l, m + log2 l) in the workspace, and
// tree_merge_kernel joins them.  Row tiles that share their keys go in twos to
// neighbouring CTAs that read the same tiles at the same time, the second from L2:
// one list of all of them read DRAM 1.8 times over and took 182 us for 4 trees of 64
// nodes behind 32768 keys (32/8 heads), against 152 (now 142).
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
// P is kept as two bf16 terms, the rounded weight and the rounded rest (together
// 17 bits), each with its PV MMA: one term's error (2^-9 of a weight) is as large
// as a bf16 output's own rounding.  fp32 rows have a third term, in shared memory,
// where a piece is short (kTrThird); in long ones the tensor cores' accumulation of
// O, which truncates, outweighs what it would mend (4e-6 of a row where pieces have
// 21 tiles, 1.6e-5 for 108).
//
// Registers are what the softmax threads are short of (128 with two CTAs per SM):
// Q goes to shared memory without them (cp.async), a warp's place in the list waits
// there while it works on a piece, and exponentials are taken where they are split.
// Spills cost more than their instructions in calls of a few tiles (their first
// touch misses): 11.4 to 10.9 us for 308 keys, 150 to 144 for the case above.
//
// What bounds it.  Few rows: HBM (8 rows of each of 8 kv heads behind 4 x 32768 keys,
// 537 MB, 91 us, 5.9 TB/s with a start and a merge of some 12).  Full row tiles: the
// MMAs' chain (scores, softmax, PV, the next scores into the same buffer), 0.75 us a
// tile alone and 1.3 us for the two CTAs of an SM together, of which the tensor
// pipe is busy 72 % (the two P terms, and score MMAs bound by shared memory at N =
// 64).  Small calls: latency, 9 us for one tile of one sequence.
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
// Two stages of each: a third of K, or of V, made no difference (within 1 % from
// one tile to 16384), as the loads run a step and a half ahead of their MMAs.
constexpr int kTrKStages = 2, kTrVStages = 2;
constexpr int kTrOffQ = 0;
constexpr int kTrOffK = kTrOffQ + 2 * kTrQHalf;
constexpr int kTrOffV = kTrOffK + kTrKStages * kTrTile;
constexpr int kTrOffP = kTrOffV + kTrVStages * kTrTile;  // third P term: 128 rows x 64 keys
constexpr int kTrOffBar = kTrOffP + kPfRows * 128;
// 8-byte slots: K full / empty and V full / empty per stage, Q, two score, two
// P and two PV barriers, the TMEM address, the abort flag, the last piece with
// a V row that is not finite, the CTA's place in the second list and, for each of
// the softmax warps, its place while it works on a piece
constexpr int kTsKFull = 0, kTsKEmpty = kTsKFull + kTrKStages, kTsVFull = kTsKEmpty + kTrKStages;
constexpr int kTsVEmpty = kTsVFull + kTrVStages, kTsQ = kTsVEmpty + kTrVStages, kTsS = kTsQ + 1;
constexpr int kTsP = kTsS + 2, kTsO = kTsP + 2, kTsTmem = kTsO + 2, kTsAbort = kTsTmem + 1;
constexpr int kTsBad = kTsAbort + 1, kTsPlace = kTsBad + 1, kTsSlots = 48;
constexpr int kTrSmem = kTrOffBar + kTsSlots * 8;
static_assert(2 * (kTrSmem + 1024) <= 228 * 1024, "two CTAs do not fit an SM");
constexpr int kTrCols = 256;    // tensor memory columns: S_0 0.., S_1 64.., O 128..
constexpr int kTrSCols = 64, kTrO = 128;

// A piece's start and end (Q, the first tile's masks, the rows' way out) cost about
// as much as this many tiles: with 2 / 4 / 5 / 6, 64 trees of up to 8 nodes behind 1 to
// 8192 keys (12/2 heads) took 27.6 / 23.5 / 24.0 / 23.4 us, six chains behind 9 to 30
// thousand (20/4 heads) 52.4 / 48.3 / 47.7 / 47.2.
constexpr int kTrPieceTiles = 5;

// fp32 rows of a piece of up to this many tiles have a third P term.  Two leave
// 2e-6 of a row, three 4e-7, while the accumulation's truncation grows by 1.3e-7 a
// tile with two and 2e-7 with three: even at 13 tiles.
constexpr int kTrThird = 12;

// What the merge has to know of CTA c's first piece, where it goes on with a unit
// that an earlier CTA began: the unit's rows, CTAs first .. last and output rows.
struct TreeCut {
  int rows, first, last;  // rows 0: the CTA starts with a unit's first tile
  int q0, g, mt, step, base;  // piece i of the unit is CTA base + step i's
};

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
  int pairs;              // splits / 2
  TreeCut *cuts;          // [2 lists][splits]
  float *part_o;          // [2 lists][2][splits][128 rows][128]
  float *part_lse;        // [2 lists][2][splits][128]
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
// Two row tiles of a (sequence, kv head) run side by side, on the two CTAs of a
// pair, so that what one reads of the cache is in L2 for the other: list 0, cut
// over the pairs, holds them, a row tile pair under its longer tile's keys.  List
// 1, cut over the CTAs, holds the row tiles that are left over.
__device__ __forceinline__ int paired(const TreeParams &p, int row_tiles) {
  return p.pairs ? row_tiles & ~1 : 0;
}
// Length of one kv head of the sequence in the lists (whose whole lengths the host
// has made sure fit an int).
__device__ __forceinline__ void head_weight(const TreeParams &p, const TreeSeq &q, int (&w)[2]) {
  w[0] = w[1] = 0;
  const int m = row_tiles(p, q), two = paired(p, m);
  for (int i = 1; i < two; i += 2) w[0] += unit_tiles(p, q, i) + kTrPieceTiles;
  for (int i = two; i < m; ++i) w[1] += unit_tiles(p, q, i) + kTrPieceTiles;
}

// A list is cut into parts of this length, while it lasts: down to a tile each, since
// tiles side by side save more than a merge of more pieces costs (parts of four
// tiles at least took 13.0 us for one sequence of 308 keys, against 11.3, 15.5 / 13.3
// for one of 2000; no difference from 600 tiles on).
__device__ __forceinline__ int part_length(int N, int parts) {
  return (int)(((unsigned)N + (unsigned)parts - 1u) / (unsigned)parts);
}
__device__ __forceinline__ int part_of(int x, int len) {
  return (int)((unsigned)x / (unsigned)len);
}

// A CTA's place in a list: the unit it is in and where that unit starts.
struct TreePlace {
  int x, end, start;
  int s, g, mt;
  TreeSeq q;
};
static_assert(5 * sizeof(TreePlace) <= (kTsSlots - kTsPlace) * 8, "the place does not fit");

struct TreePiece {
  TreeSeq q;
  int s, g, mt, t0, t1, tiles, list;
};

// The next piece of a CTA's parts of the lists; every warp runs this for itself.
struct TreeWalk {
  TreePlace at;
  const TreePlace *second;
  int list;

  __device__ __forceinline__ bool next(const TreeParams &p, TreePiece &r) {
    while (true) {
      if (at.x >= at.end) {
        if (list == 1) return false;
        list = 1;
        at = *second;
        continue;
      }
      const int m = row_tiles(p, at.q), two = paired(p, m);
      // of a pair, the first CTA's row tile may end some tiles before the second's
      const int span = unit_tiles(p, at.q, list == 0 ? at.mt + 1 : at.mt);
      const int mt = list == 0 ? at.mt + (int)(blockIdx.x & 1) : at.mt;
      const int tiles = unit_tiles(p, at.q, mt);
      const int rel = at.x - at.start;
      const bool got = rel < tiles;
      if (got) {
        r.q = at.q;
        r.s = at.s;
        r.g = at.g;
        r.mt = mt;
        r.tiles = tiles;
        r.t0 = rel;
        r.t1 = min(tiles, at.end - at.start);
        r.list = list;
      }
      at.start += span + kTrPieceTiles;
      at.x = at.start;
      at.mt += list == 0 ? 2 : 1;
      if (at.mt == (list == 0 ? two : m)) {
        if (++at.g == p.hkv) {
          at.g = 0;
          if (at.x < at.end) at.s = next_seq(p, at.s, list, at.q);
        }
        at.mt = list == 0 ? 0 : paired(p, row_tiles(p, at.q));
      }
      if (got) return true;
    }
  }
  // The next sequence with something in the list (there is one).
  __device__ __forceinline__ static int next_seq(const TreeParams &p, int s, int list,
                                                 TreeSeq &q) {
    bool some;
    do {
      q = tree_seq(p, ++s, false);
      const int m = row_tiles(p, q), two = paired(p, m);
      some = list == 0 ? two > 0 : two < m;
    } while (!some && s + 1 < p.num_seqs);
    return s;
  }
};

// The CTA's parts of the lists (places without work: x = end).  Every warp works it
// out for itself, a lane per run of sequences.
__device__ __forceinline__ void tree_plan(const TreeParams &p, TreePlace (&places)[2],
                                          int (&len)[2]) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int per = (int)(((unsigned)p.num_seqs + 31u) / 32u);
  const int s0 = min(p.num_seqs, lane * per), s1 = min(p.num_seqs, s0 + per);
  int mine[2] = {0, 0}, upto[2], w[2];
  TreeSeq q = {0, 0, 0};
  for (int s = s0; s < s1; ++s) {
    q = tree_seq(p, s, blockIdx.x == 0 && threadIdx.x < 32);
    head_weight(p, q, w);
    mine[0] += w[0] * p.hkv;
    mine[1] += w[1] * p.hkv;
  }
  upto[0] = mine[0];
  upto[1] = mine[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(kAll, upto[0], o), b = __shfl_up_sync(kAll, upto[1], o);
    if (lane >= o) {
      upto[0] += a;
      upto[1] += b;
    }
  }
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    const int N = __shfl_sync(kAll, upto[l], 31);
    const int part = l == 0 ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int parts = l == 0 ? p.pairs : p.splits;
    TreePlace &r = places[l];
    r.x = r.end = 0;
    len[l] = 1;
    if (N == 0 || part >= parts) continue;
    len[l] = part_length(N, parts);
    if (part > (N - 1) / len[l]) continue;
    const int x0 = part * len[l];
    const unsigned has = __ballot_sync(kAll, x0 >= upto[l] - mine[l] && x0 < upto[l]);
    int v[8] = {};
    if ((has >> lane) & 1u) {
      int at = upto[l] - mine[l];
      for (int s = s0; s < s1; ++s) {
        if (per > 1) q = tree_seq(p, s, false);
        head_weight(p, q, w);
        if (x0 >= at + w[l] * p.hkv) {
          at += w[l] * p.hkv;
          continue;
        }
        int g = 0, mt = l == 0 ? 0 : paired(p, row_tiles(p, q));
        while (x0 >= at + w[l]) {
          at += w[l];
          ++g;
        }
        while (true) {
          const int unit = unit_tiles(p, q, mt + 1 - l) + kTrPieceTiles;
          if (x0 < at + unit) break;
          at += unit;
          mt += 2 - l;
        }
        v[0] = at, v[1] = s, v[2] = g, v[3] = mt, v[4] = q.q0, v[5] = q.nodes, v[6] = q.keys;
        break;
      }
    }
    const int from = __ffs(has) - 1;
    r.x = x0;
    r.end = min(N, x0 + len[l]);
    r.start = __shfl_sync(kAll, v[0], from);
    r.s = __shfl_sync(kAll, v[1], from);
    r.g = __shfl_sync(kAll, v[2], from);
    r.mt = __shfl_sync(kAll, v[3], from);
    r.q.q0 = __shfl_sync(kAll, v[4], from);
    r.q.nodes = __shfl_sync(kAll, v[5], from);
    r.q.keys = __shfl_sync(kAll, v[6], from);
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

// A store without a branch around it.
__device__ __forceinline__ void store_if(bool yes, char *to, const uint4 &v) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
      "@p st.global.v4.u32 [%1], {%2, %3, %4, %5};\n\t}" ::"r"((int)yes),
      "l"(__cvta_generic_to_global(to)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
      : "memory");
}
__device__ __forceinline__ void store_if(bool yes, char *to, uint32_t a, uint32_t b) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
      "@p st.global.v2.u32 [%1], {%2, %3};\n\t}" ::"r"((int)yes),
      "l"(__cvta_generic_to_global(to)), "r"(a), "r"(b)
      : "memory");
}

// Clears, in a staged V tile, the rows of keys from `end` on and the elements of keys
// from `done` on that are not finite (then *bad = piece).  Thread r of 128 has the
// 16-byte chunk r % 16 of keys r / 16 + 8 k.  0 x is NaN exactly where x is not
// finite, so a sum of such products tells.
__device__ __forceinline__ void clean_v(uint32_t tile, int r, int key0, int done, int end,
                                        volatile int *bad, int piece) {
  const int ch = r & 15, k0 = r >> 4;
  const uint32_t at = tile + (ch >> 3) * kTrHalf + sw128(k0, ch & 7);  // (+ 1024 a step: k % 8)
  uint4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    const int key = key0 + k0 + 8 * k;
    if (key >= done && key < end) v[k] = lds128(at + 1024 * k);
    if (key >= end)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + 1024 * k), "r"(0u)
                   : "memory");
  }
  uint32_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[0]) : "r"(v[k].x), "r"(0u));
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[1]) : "r"(v[k].y), "r"(0u));
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[2]) : "r"(v[k].z), "r"(0u));
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[3]) : "r"(v[k].w), "r"(0u));
  }
  if (((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0u) {  // rare
    *bad = piece;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const int key = key0 + k0 + 8 * k;
      if (key < done || key >= end) continue;
      uint4 x = lds128(at + 1024 * k);
      uint32_t *w = &x.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
      }
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + 1024 * k), "r"(x.x),
                   "r"(x.y), "r"(x.z), "r"(x.w)
                   : "memory");
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <bool kF32>  // fp32 rows, else bf16
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
  TreePlace *second = reinterpret_cast<TreePlace *>(bars + kTsPlace);

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
  TreeWalk walk;
  walk.second = second;
  walk.list = 0;
  {
    TreePlace places[2];
    int len[2];
    tree_plan(p, places, len);
    walk.at = places[0];
    if (tid == 0) *second = places[1];
    if (warp == 3 && lane == 0) {
      // what the merge has to know of a part that goes on with a unit
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        const TreePlace &at = places[l];
        TreeCut cut = {};
        if (at.x < at.end && at.x > at.start) {
          const int mt = l == 0 ? at.mt + (int)(blockIdx.x & 1) : at.mt;
          const int tiles = unit_tiles(p, at.q, mt);
          if (at.x - at.start < tiles) {
            cut.rows = min(kPfRows, at.q.nodes * p.group - mt * kPfRows);
            cut.first = part_of(at.start, len[l]);
            cut.last = part_of(at.start + tiles - 1, len[l]);
            cut.q0 = at.q.q0;
            cut.g = at.g;
            cut.mt = mt;
            cut.step = 2 - l;
            cut.base = l == 0 ? (int)(blockIdx.x & 1) : 0;
          }
        }
        p.cuts[l * p.splits + blockIdx.x] = cut;
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + kTrO;
  if ((base & 1023) != 0) {  // (the swizzle needs it; without static shared memory it is so)
    if (tid == 0) report(p.err, PA_DEVERR_WAIT_TIMEOUT);
    walk.at.x = walk.at.end;
    walk.list = 1;
  }
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
#pragma unroll 1
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
      const bool third = kF32 && n <= kTrThird;
#pragma unroll 1
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
          if (third) {
#pragma unroll
            for (int ks = 0; ks < kPfKeys / 16; ++ks)
              umma_f16_ss(tmem_o, umma_desc(base + kTrOffP + ks * 32, 16, 1024),
                          umma_desc(vb + ks * 16 * 128, kTrHalf, 1024), idesc_pv, 1u);
          }
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
    TreePlace *const save = second + 1 + (warp & 3);
    while (ok && walk.next(p, u)) {
      if (lane == 0) *save = walk.at;  // (registers are short in between)
      const int R = u.mt * kPfRows + r, limit = u.q.nodes * p.group;
      const bool valid = R < limit;
      const bool alive = u.mt * kPfRows + lb < limit;  // any row of the warp
      const int node = by_group(p, R);
      const int done = u.q.keys - u.q.nodes;
      // this lane's row of q and out (T * Hq < 2^32); another lane's comes by shuffle
      const uint32_t my_row = (uint32_t)(u.q.q0 + node) * (uint32_t)p.hq +
                              (uint32_t)(u.g * p.group + R - node * p.group);
      // parents of the window first .. first + 63 of nodes, two a lane
      const int32_t *par = p.parents + u.q.q0;
      auto parent = [&](int n) { return n >= 0 && n < u.q.nodes ? par[n] : -1; };
      int par0 = -1, par1 = -1;
      if (alive && (u.t1 - 1) * kPfKeys > done - kPfKeys) {
        const int first = (u.t1 - 1) * kPfKeys - done;
        par0 = parent(first + lane);
        par1 = parent(first + lane + 32);
      }
      // Q rows, half a warp a row, into the layout the TMA gives K tiles
      if (alive) {
        const int ch = lane & 15;
        const uint32_t a0 = base + kTrOffQ + (ch >> 3) * kTrQHalf + lb * 128;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 2 * i + (lane >> 4);
          const bool there = u.mt * kPfRows + lb + x < limit;
          const uint32_t from = __shfl_sync(kAll, my_row, x), row = there ? from : 0u;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(a0 + sw128(x, ch & 7)),
                       "l"(p.q + (size_t)row * kHeadDim + 8 * ch), "r"(there ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (p.q_and != 0xffffffffu || p.q_xor != 0u) {  // a scale <= 0, folded into q
          for (int i = 0; i < 16; ++i) {
            const uint32_t a = a0 + sw128(2 * i + (lane >> 4), ch & 7);
            const uint4 v = lds128(a);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a),
                         "r"((v.x & p.q_and) ^ p.q_xor), "r"((v.y & p.q_and) ^ p.q_xor),
                         "r"((v.z & p.q_and) ^ p.q_xor), "r"((v.w & p.q_and) ^ p.q_xor)
                         : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      mbar_arrive(b_q);
      // m: the reference of this row's exponentials (base 2); it moves only when
      // a tile's largest exceeds it by more than 8, so P <= 256 and O is rescaled
      // rarely.  l: the row's sum.  up: the next node of the walk to the root.
      float m = -INFINITY, l = 0.f;
      const bool third = kF32 && u.t1 - u.t0 <= kTrThird;
      // A tile's 64 keys are a window of 64 nodes, whose parents the warp holds,
      // two a lane: a step of the walk is a shuffle.
      int up = valid ? node : -1;
      auto climb = [&](int first, int par0, int par1, uint32_t (&vis)[2]) {
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
      if (alive && (u.t1 - 1) * kPfKeys > done - kPfKeys) {  // the windows above the piece's last tile
        uint32_t unused[2] = {0u, 0u};
        const int top = by_group(p, min(u.mt * kPfRows + lb + 31, limit - 1));
        for (int j = (done + top) / kPfKeys; j >= u.t1; --j) {
          const int first = j * kPfKeys - done;
          climb(first, parent(first + lane), parent(first + lane + 32), unused);
        }
      }
#pragma unroll 1
      for (int j = u.t1 - 1; j >= u.t0 && ok; --j, ++it) {
        const int st = it % kTrVStages, buf = it & 1;
        const int key0 = j * kPfKeys;
        const bool in_tree = key0 > done - kPfKeys;  // the tile holds drafted nodes
        uint32_t vis[2] = {0u, 0u};
        if (in_tree && alive) {
          climb(key0 - done, par0, par1, vis);
          par0 = parent(key0 - kPfKeys - done + lane);
          par1 = parent(key0 - kPfKeys - done + lane + 32);
          if (valid && key0 < done) {
            const int below = done - key0;  // 1 .. 63 committed keys
            vis[0] |= below >= 32 ? 0xffffffffu : (1u << below) - 1u;
            vis[1] |= below > 32 ? (1u << (below - 32)) - 1u : 0u;
          }
        }
        // V rows of the tile that some rows may not see: those past the end may
        // hold anything and are cleared; a drafted node's infinities and NaN are
        // cleared here and put into the rows that see it at the end
        if (in_tree) {
          ok = __all_sync(kAll, mbar_wait(b_v_full + 8 * st, (it / kTrVStages) & 1, abort_flag,
                                          p.err));
          if (!ok) break;
          clean_v(base + kTrOffV + st * kTrTile, r, key0, done, u.q.keys, bad_piece, piece);
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
          const float neg_m = m == -INFINITY ? 0.f : -m;
          const uint64_t c2 = pack_f32x2(c, c), nm2 = pack_f32x2(neg_m, neg_m);
          if (third && it > 0) {  // the third term's place is read until the PV before is over
            ok = __all_sync(kAll, mbar_wait(b_o + 8 * ((it - 1) & 1), ((it - 1) >> 1) & 1,
                                            abort_flag, p.err));
            if (!ok) break;
          }
          // P over the scores: hi parts (two keys a column) in the buffer's
          // columns 0 .. 31, lo parts in 32 .. 63
          uint64_t ps4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x0, x1;
              unpack_f32x2(fma_f32x2(pack_f32x2(sv[cc >> 1][16 * (cc & 1) + 2 * i],
                                                sv[cc >> 1][16 * (cc & 1) + 2 * i + 1]),
                                     c2, nm2),
                           x0, x1);
              const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
              hi[i] = float2_to_bf16x2(e0, e1);
              const uint64_t e2 = pack_f32x2(e0, e1);
              ps4[i & 3] = add_f32x2(ps4[i & 3], e2);
              float d0, d1;
              unpack_f32x2(sub_f32x2(e2, pack_f32x2(__uint_as_float(hi[i] << 16),
                                                    __uint_as_float(hi[i] & 0xFFFF0000u))),
                           d0, d1);
              lo[i] = float2_to_bf16x2(d0, d1);
            }
            tmem_st8(sb + trow + cc * 8, hi);
            tmem_st8(sb + trow + kTrSCols / 2 + cc * 8, lo);
            if (third) {  // 16 keys of the row (the weights again: keeping them spills)
              uint32_t low[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float x0, x1;
                unpack_f32x2(fma_f32x2(pack_f32x2(sv[cc >> 1][16 * (cc & 1) + 2 * i],
                                                  sv[cc >> 1][16 * (cc & 1) + 2 * i + 1]),
                                       c2, nm2),
                             x0, x1);
                low[i] = float2_to_bf16x2(
                    (ex2_approx(x0) - __uint_as_float(hi[i] << 16)) - __uint_as_float(lo[i] << 16),
                    (ex2_approx(x1) - __uint_as_float(hi[i] & 0xFFFF0000u)) -
                        __uint_as_float(lo[i] & 0xFFFF0000u));
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 base + kTrOffP + sw128(r, 2 * cc + h)),
                             "r"(low[4 * h]), "r"(low[4 * h + 1]), "r"(low[4 * h + 2]),
                             "r"(low[4 * h + 3])
                             : "memory");
              }
            }
          }
          float ps8[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) unpack_f32x2(ps4[x], ps8[2 * x], ps8[2 * x + 1]);
          l = l * alpha + (((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) +
                           ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7])));
          tmem_wait_st();
          if (third) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
        const long long slot = ((2 * u.list + (u.t0 == 0)) * (long long)p.splits + blockIdx.x) *
                                   kPfRows + lb;
        // 32 columns of the warp's rows at a time go through its own Q rows (which
        // no MMA reads any more), so that eight lanes store a row's 128 bytes
        const uint32_t stage = base + kTrOffQ + lb * 128;
        const bool narrow = whole && !kF32;
        char *to = whole ? static_cast<char *>(p.out)
                         : reinterpret_cast<char *>(p.part_o + slot * kHeadDim);
        uint32_t rows[8];  // of this lane's stores
        const int left = limit - (u.mt * kPfRows + lb + (lane >> 3));  // row 4 i is one: 4 i < left
#pragma unroll
        for (int i = 0; i < 8; ++i)
          rows[i] = __shfl_sync(kAll, whole ? my_row : (uint32_t)lane, 4 * i + (lane >> 3));
        to += (size_t)(lane & 7) * (narrow ? 8 : 16);
#pragma unroll 1
        for (int cc = 0; cc < kHeadDim / 32; ++cc) {
          uint32_t dims = 0;
          if (valid && bad)
            dims = not_finite(p, u.s, u.q.q0, done, u.g, node, u.t0 * kPfKeys,
                              (u.t1 - 1) * kPfKeys + (kPfKeys - 1), cc);
          __syncwarp();
          float ov[32];
          tmem_ld32(tmem_o + trow + cc * 32, ov);
          if (dims != 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((dims >> i) & 1u) ov[i] = __int_as_float(0x7fffffff);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + sw128(lane, i)),
                         "f"(ov[4 * i] * inv), "f"(ov[4 * i + 1] * inv), "f"(ov[4 * i + 2] * inv),
                         "f"(ov[4 * i + 3] * inv));
          __syncwarp();
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "r"(stage + sw128(4 * i + (lane >> 3), lane & 7)));
          __syncwarp();
          if (narrow) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              store_if(4 * i < left, to + (size_t)rows[i] * 256 + cc * 64,
                       float2_to_bf16x2(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                       float2_to_bf16x2(__uint_as_float(w[i].z), __uint_as_float(w[i].w)));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              store_if(4 * i < left, to + (size_t)rows[i] * 512 + cc * 128, w[i]);
          }
        }
        __syncwarp();
        if (valid && !whole)
          p.part_lse[slot + lane] = l == 0.f ? -INFINITY : m + log2f(l);
      }
      tc_fence_before();
      __syncwarp();
      walk.at = *save;
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
// where a CTA has few rows; a warp has eight loads of 512 bytes in flight, of one
// row or, where a row has few pieces, of four or two.
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

// Pieces x .. x + kPieces - 1 (below cb) of kRows rows (below 0: none), all loads first.
template <int kRows, int kPieces>
__device__ __forceinline__ void add_pieces(const TreeParams &p, const TreeCut &cut, int list,
                                           const int (&row)[kRows], int x, int cb,
                                           RowSum *const (&a)[kRows]) {
  const int lane = threadIdx.x & 31;
  float lse[kRows][kPieces];
  float4 o[kRows][kPieces];
#pragma unroll
  for (int k = 0; k < kRows; ++k)
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      lse[k][i] = -INFINITY;
      o[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row[k] >= 0 && x + i < cb) {
        const long long slot = ((2 * list + (x + i == cut.first)) * (long long)p.splits +
                                cut.base + (long long)cut.step * (x + i)) * kPfRows + row[k];
        lse[k][i] = p.part_lse[slot];
        o[k][i] = reinterpret_cast<const float4 *>(p.part_o + slot * kHeadDim)[lane];
      }
    }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    RowSum &s = *a[k];
    float top = s.m;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) top = fmaxf(top, lse[k][i]);
    const float ref = top == -INFINITY ? 0.f : top;  // nothing seen so far: weights zero
    const float old = exp2f(s.m - ref);
    s.w *= old;
    s.o.x *= old, s.o.y *= old, s.o.z *= old, s.o.w *= old;
    s.m = top;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const float w = exp2f(lse[k][i] - ref);
      if (!(w == 0.f)) row_add(s, w, o[k][i]);
    }
  }
}

__device__ __forceinline__ void write_row(const TreeParams &p, const TreeCut &cut, int r,
                                          const RowSum &a) {
  const float inv = a.w > 0.f ? 1.f / a.w : a.w;
  const int R = cut.mt * kPfRows + r, node = by_group(p, R);
  const long long at = ((long long)(cut.q0 + node) * p.hq + cut.g * p.group +
                        (R - node * p.group)) * kHeadDim + (threadIdx.x & 31) * 4;
  const float4 o = make_float4(a.o.x * inv, a.o.y * inv, a.o.z * inv, a.o.w * inv);
  if (p.out_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = o;
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
        make_uint2(float2_to_bf16x2(o.x, o.y), float2_to_bf16x2(o.z, o.w));
}

// The CTA's rows, kRows at a time by a warp, of kPieces pieces at most.
template <int kRows, int kPieces>
__device__ __forceinline__ void merge_rows(const TreeParams &p, const TreeCut &cut, int list,
                                           int n, int i0,
                                           int rows, int warp) {
  for (int k = warp * kRows; k < rows; k += kTmWarps * kRows) {
    int row[kRows];
    RowSum s[kRows], *to[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = i0 + (k + j) * n;
      row[j] = k + j < rows && r < cut.rows ? r : -1;
      s[j] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      to[j] = &s[j];
    }
    add_pieces<kRows, kPieces>(p, cut, list, row, cut.first, cut.last + 1, to);
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (row[j] >= 0) write_row(p, cut, row[j], s[j]);
  }
}

__device__ __forceinline__ void merge_cut(const TreeParams &p, const TreeCut &cut, int list) {
  __shared__ float share_m[kTmWarps], share_w[kTmWarps];
  __shared__ float4 share_o[kTmWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = cut.last - cut.first;
  const int i0 = (int)blockIdx.x / cut.step - cut.first - 1;
  const int rows = (cut.rows - i0 + n - 1) / n;  // rows of this CTA
  // warps that share a row
  const int share = rows > kTmWarps / 2 ? 1 : rows > kTmWarps / 4 ? 2 : rows > kTmWarps / 8 ? 4
                    : rows > kTmWarps / 16 ? 8 : kTmWarps;
  const int each = (n + share) / share;  // pieces of a warp
  const int ca = cut.first + (warp % share) * each, cb = min(cut.last + 1, ca + each);
  if (share == 1 && each <= 4) {
    if (each <= 2)
      merge_rows<4, 2>(p, cut, list, n, i0, rows, warp);
    else
      merge_rows<2, 4>(p, cut, list, n, i0, rows, warp);
    return;
  }
  for (int k = 0; k < rows; k += kTmWarps / share) {
    const int r = i0 + (k + warp / share) * n;
    const bool mine = r < cut.rows;
    RowSum a = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (mine)
      for (int x = ca; x < cb; x += 8) {
        const int row[1] = {r};
        RowSum *one[1] = {&a};
        add_pieces<1, 8>(p, cut, list, row, x, cb, one);
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
    write_row(p, cut, r, a);
  }
}

__global__ void __launch_bounds__(32 * kTmWarps) tree_merge_kernel(const TreeParams p) {
  griddep_wait();
  griddep_launch_dependents();
  {
    const int list = blockIdx.y;
    const TreeCut cut = p.cuts[list * p.splits + blockIdx.x];
    if (cut.rows) merge_cut(p, cut, list);
  }
}

constexpr size_t kTrHead = 256;  // the error word
size_t tree_part_bytes(long long splits) {
  return (size_t)splits * 4 * kPfRows * kHeadDim * sizeof(float);
}
size_t tree_lse_bytes(long long splits) { return (size_t)splits * 4 * kPfRows * sizeof(float); }
size_t tree_workspace(long long splits) {
  return kTrHead + tree_part_bytes(splits) + tree_lse_bytes(splits) +
         (size_t)splits * 2 * sizeof(TreeCut);
}

template <bool kF32>
cudaError_t launch_tree(const CUtensorMap &tk, const CUtensorMap &tv, const TreeParams &p,
                        int device, cudaStream_t s) {
  static std::atomic<bool> configured[64] = {};
  const cudaError_t e = set_smem_once(configured, tree_kernel<kF32>, device, kTrSmem);
  if (e != cudaSuccess) return e;
  // two CTAs per SM: all of the unified L1 / shared memory as shared memory (a hint)
  cudaFuncSetAttribute(tree_kernel<kF32>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  return launch_kernel(tree_kernel<kF32>, dim3((unsigned)p.splits), dim3(kTrThreads), kTrSmem, s,
                       true, tk, tv, p);
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
  // the lists' lengths fit an int, whatever the lengths on the device
  const long long most_tiles = (long long)block_table_stride * kBlockSize / kPfKeys + 2;
  const long long most_nodes = max_q_len < total_tokens ? max_q_len : total_tokens;
  const long long rows = (most_nodes * (num_q_heads / num_kv_heads) + kPfRows - 1) / kPfRows;
  if (most_tiles + kTrPieceTiles > (1ll << 31) / num_kv_heads / rows / num_seqs)
    return PA_ERR_UNSUPPORTED;
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
  p.pairs = splits / 2;
  p.part_o = reinterpret_cast<float *>(ws + kTrHead);
  p.part_lse = reinterpret_cast<float *>(ws + kTrHead + tree_part_bytes(splits));
  p.cuts = reinterpret_cast<TreeCut *>(ws + kTrHead + tree_part_bytes(splits) +
                                       tree_lse_bytes(splits));
  p.err = static_cast<int32_t *>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p.out_f32 ? launch_tree<true>(tk, tv, p, device, s)
                                  : launch_tree<false>(tk, tv, p, device, s);
  if (e != cudaSuccess) return PA_ERR_LAUNCH;
  if (splits > 1 &&
      launch_kernel(tree_merge_kernel, dim3((unsigned)splits, 2), dim3(32 * kTmWarps), 0, s, true,
                    p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}
