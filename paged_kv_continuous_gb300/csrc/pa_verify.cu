// pa_verify_tree: the walk down a tree of drafted tokens, and the token after it.
//
// With p and q the target's and the draft's row at the node where the walk
// stands, every rejected child replaces the target by the normalised positive
// part of (target - draft).  Those steps collapse: if the target is max(p - beta
// q, 0) / W, then after rejecting a draw from s q it is max(p - (beta + s W) q, 0)
// / W', because what is zero stays zero.  So one number carries all rejections,
// a test needs two elements of the rows, and only a rejection and the last draw
// need a pass over them, for the weights' sum.
//
// A cluster of CTAs takes a sequence.  Each warp owns a contiguous segment of
// the vocabulary; a pass leaves every segment's sum with every CTA (through
// distributed shared memory, one cluster barrier), so that all CTAs take the same
// decisions, and the last draw looks for its segment among them and scans that
// one alone.  Elements that a test may need are loaded for all nodes at once,
// ahead of the walk.
//
// A drawn token is a whole number next to a border of the running sum, so the
// sums carry more than fp32: a weight is an unevaluated pair of floats (the
// product's and the difference's rounding errors kept), and pairs are added into
// pairs, in lanes, warps and over the segments, some 20 fp32 operations an
// element.  The tests of single nodes are taken in pairs too (their products are
// exact).  fp64, whose rate on this chip is low, took 61 us where 64 sequences of
// 32000 tokens joined lanes and segments in it (now 8), and 1 to 2 us of a rejection
// where a node's test was in it.
//
// Bound by latency for few sequences, and by HBM for many: a pass reads 8 bytes
// an element.
#include <climits>

#include <cooperative_groups.h>

#include "pa_common.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kVfThreads = 256, kVfWarps = kVfThreads / 32;
constexpr int kVfNodes = 256;          // nodes whose elements are held at a time
constexpr int kVfMaxVocab = 1 << 20;   // (a bit for each token, in shared memory)
constexpr float kVfLeast = 1.f / (1 << 24);

struct VerifyParams {
  int32_t *accepted, *path, *out_tokens;
  const int32_t *tokens, *parents, *cu;
  int num_seqs, total, width;
  const float *p;
  long long p_stride;
  const float *q;
  long long q_stride;
  int vocab;
  const float *u, *u_last;
  int again;    // siblings drawn with replacement
  int segment;  // tokens of a warp, a multiple of 128
  int32_t *err;
};

// hi + lo, with hi the sum's rounding to a float.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ bool above(const Pair &a, const Pair &b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
// The sum, within 2^-46 of it where both are positive.  The order of the two does
// not matter.
__device__ __forceinline__ Pair plus(const Pair &a, const Pair &b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  const float e = ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo);
  const float hi = s + e;
  return {hi, e - (hi - s)};
}
__device__ __forceinline__ Pair minus(const Pair &a, const Pair &b) {
  return plus(a, {-b.hi, -b.lo});
}
// a b and a / b, within 2^-44.
__device__ __forceinline__ Pair times(const Pair &a, const Pair &b) {
  const float h = __fmul_rn(a.hi, b.hi);
  const float l = fmaf(a.hi, b.hi, -h) + fmaf(a.hi, b.lo, a.lo * b.hi);
  const float hi = h + l;
  return {hi, l - (hi - h)};
}
__device__ __forceinline__ Pair over(const Pair &a, const Pair &b) {
  const float x = a.hi / b.hi;
  const Pair rest = minus(a, times({x, 0.f}, b));
  return plus({x, 0.f}, {rest.hi / b.hi, 0.f});
}
__device__ __forceinline__ Pair shfl_up(const Pair &a, int by) {
  return {__shfl_up_sync(0xffffffffu, a.hi, by), __shfl_up_sync(0xffffffffu, a.lo, by)};
}
__device__ __forceinline__ Pair shfl(const Pair &a, int lane) {
  return {__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
// Sums over the lanes up to this one.
__device__ __forceinline__ Pair warp_upto(Pair x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = shfl_up(x, o), z = plus(x, y);
    if ((int)(threadIdx.x & 31) >= o) x = z;
  }
  return x;
}

// max(p - beta q, 0) as a pair, beta = bh + bl.
__device__ __forceinline__ Pair weight(float p, float q, float bh, float bl) {
  const float ph = __fmul_rn(q, bh);
  const float pl = fmaf(q, bl, fmaf(q, bh, -ph));
  // p - ph = s + ((p - s) - ph) where p >= ph; elsewhere nothing is left anyway
  const float s = __fadd_rn(p, -ph);
  const float lo = ((p - s) - ph) - pl;
  const float hi = s + lo;
  return {hi > 0.f ? hi : 0.f, hi > 0.f ? lo - (hi - s) : 0.f};
}

// Two running sums side by side, two floats an instruction: hi's, and what adding
// to them lost.
struct Sum2 {
  uint64_t hi, lo;
};
__device__ __forceinline__ void add2(Sum2 &a, uint64_t x) {
  const uint64_t s = add_f32x2(a.hi, x), b = sub_f32x2(s, a.hi);
  a.lo = add_f32x2(a.lo, add_f32x2(sub_f32x2(a.hi, sub_f32x2(s, b)), sub_f32x2(x, b)));
  a.hi = s;
}
// The weights of two tokens, as weight() takes them, added.
__device__ __forceinline__ void add_weights2(Sum2 &a, uint64_t p, uint64_t q, uint64_t bh,
                                             uint64_t bl) {
  const uint64_t ph = mul_f32x2(q, bh);
  const uint64_t minus = ph ^ 0x8000000080000000ull;
  const uint64_t pl = fma_f32x2(q, bl, fma_f32x2(q, bh, minus));
  const uint64_t s = add_f32x2(p, minus);
  const uint64_t lo = sub_f32x2(add_f32x2(sub_f32x2(p, s), minus), pl);
  float s0, s1, l0, l1, h0, h1;
  unpack_f32x2(add_f32x2(s, lo), h0, h1);
  unpack_f32x2(s, s0, s1);
  unpack_f32x2(lo, l0, l1);
  add2(a, pack_f32x2(h0 > 0.f ? s0 : 0.f, h1 > 0.f ? s1 : 0.f));
  a.lo = add_f32x2(a.lo, pack_f32x2(h0 > 0.f ? l0 : 0.f, h1 > 0.f ? l1 : 0.f));
}

// The rows of a node and the scalars of its weights.
struct Rows {
  const float *p, *q;  // q null: weights are p's
  float bh, bl;
};

// Elements i .. i + 3 of a row, of which the first n are read and the others zero.
template <bool kVec>
__device__ __forceinline__ void load4(const float *row, int i, int n, float (&v)[4]) {
  if constexpr (kVec) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n >= 4) {
      x = *reinterpret_cast<const float4 *>(row + i);
    } else {
      if (n > 0) x.x = row[i];
      if (n > 1) x.y = row[i + 1];
      if (n > 2) x.z = row[i + 2];
    }
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < n ? row[i + k] : 0.f;
  }
}
// Their weights; a bit of `out` (where there are such) marks a rejected guess.
__device__ __forceinline__ void weights4(const Rows &r, const float (&p)[4], const float (&q)[4],
                                         const uint32_t *out, int i, Pair (&w)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (r.q) {
      w[k] = weight(p[k], q[k], r.bh, r.bl);
    } else {
      const bool pos = p[k] > 0.f && !(out && ((out[(i + k) >> 5] >> ((i + k) & 31)) & 1u));
      w[k] = {pos ? p[k] : 0.f, 0.f};
    }
  }
}

// The sum of a warp's segment [s0, s1): a lane's four tokens of every 128.
// kAhead: rows of 128 tokens whose loads are in flight.
template <bool kVec, bool kDraft, int kAhead>
__device__ __forceinline__ Pair segment_sum_of(const Rows &r, int s0, int s1,
                                               const uint32_t *out) {
  const int lane = threadIdx.x & 31;
  Sum2 acc[2] = {{0, 0}, {0, 0}};
  const uint64_t bh = pack_f32x2(r.bh, r.bh), bl = pack_f32x2(r.bl, r.bl);
  const Rows plain{r.p, nullptr, 0.f, 0.f};
  for (int b = s0; b < s1; b += 128 * kAhead) {
    const int i0 = b + 4 * lane;
    float p[kAhead][4], q[kAhead][4];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + 128 * a;
      load4<kVec>(r.p, i, s1 - i, p[a]);
      if (kDraft) load4<kVec>(r.q, i, s1 - i, q[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (b + 128 * a >= s1) continue;
      if constexpr (kDraft) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          add_weights2(acc[k], pack_f32x2(p[a][2 * k], p[a][2 * k + 1]),
                       pack_f32x2(q[a][2 * k], q[a][2 * k + 1]), bh, bl);
      } else {
        Pair w[4];
        weights4(plain, p[a], q[a], out, i0 + 128 * a, w);
#pragma unroll
        for (int k = 0; k < 2; ++k) add2(acc[k], pack_f32x2(w[2 * k].hi, w[2 * k + 1].hi));
      }
    }
  }
  Pair part[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    unpack_f32x2(acc[k].hi, part[2 * k].hi, part[2 * k + 1].hi);
    unpack_f32x2(acc[k].lo, part[2 * k].lo, part[2 * k + 1].lo);
  }
  Pair sum = plus(plus(part[0], part[1]), plus(part[2], part[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    sum = plus(sum, {__shfl_xor_sync(0xffffffffu, sum.hi, o),
                     __shfl_xor_sync(0xffffffffu, sum.lo, o)});
  return sum;
}
template <bool kVec, int kAhead>
__device__ __forceinline__ Pair segment_sum(const Rows &r, int s0, int s1, const uint32_t *out) {
  return r.q ? segment_sum_of<kVec, true, kAhead>(r, s0, s1, out)
             : segment_sum_of<kVec, false, 8>(r, s0, s1, out);
}

// The first token of segment [s0, s1) where `before` plus the running sum is over
// `target`; its last of positive weight if there is none (-1: no such).  The whole
// CTA looks, a warp at 128 tokens: rows holds their sums, best what was found.
template <bool kVec>
__device__ int segment_find(const Rows &r, int s0, int s1, const uint32_t *out, Pair before,
                            const Pair &target, Pair *rows, int *best) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    best[0] = INT_MAX;
    best[1] = -1;
  }
  for (int b = s0; b < s1; b += 128 * kVfWarps) {
    const int i = b + 128 * warp + 4 * lane;
    float p[4], q[4];
    Pair w[4], c[4];
    load4<kVec>(r.p, i, s1 - i, p);
    if (r.q) load4<kVec>(r.q, i, s1 - i, q);
    weights4(r, p, q, out, i, w);
    c[0] = w[0];
    int last = -1;
#pragma unroll
    for (int k = 1; k < 4; ++k) c[k] = plus(c[k - 1], w[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (w[k].hi > 0.f) last = i + k;
    const Pair upto = warp_upto(c[3]);
    if (lane == 31) rows[warp] = upto;
    __syncthreads();
    // the rows before this one, and all of them
    const Pair sums = warp_upto(lane < kVfWarps ? rows[lane] : Pair{0.f, 0.f});
    Pair base = shfl(sums, max(warp - 1, 0));
    if (warp == 0) base = {0.f, 0.f};
    const Pair here = plus(before, base);
    Pair mine = shfl_up(upto, 1);
    mine = lane == 0 ? here : plus(here, mine);
    int found = INT_MAX;
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (w[k].hi > 0.f && above(plus(mine, c[k]), target)) found = i + k;
    found = __reduce_min_sync(0xffffffffu, found);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
      if (found != INT_MAX) atomicMin(best, found);
      if (last >= 0) atomicMax(best + 1, last);
    }
    before = plus(before, shfl(sums, 31));
    __syncthreads();
    if (best[0] != INT_MAX) break;
  }
  return best[0] != INT_MAX ? best[0] : best[1];
}

// All segments' sums into `sums` of every CTA of the cluster.  Alternate passes use
// alternate halves of `mine`: a CTA still reads one pass's while another writes the
// next one's, and the pass after that waits for it at the barrier between.
template <bool kVec, int kRanks, int kAhead>
__device__ void sum_rows(cg::cluster_group &cluster, const Rows &r, const uint32_t *out, int s0,
                         int s1, Pair (&mine)[2][kVfWarps], Pair *sums, int pass) {
  const int tid = threadIdx.x, warp = tid >> 5;
  const Pair sum = segment_sum<kVec, kAhead>(r, s0, s1, out);
  if ((tid & 31) == 0) mine[pass & 1][warp] = sum;
  cluster.sync();
  if (tid < kRanks * kVfWarps) {
    const int from = tid / kVfWarps;
    sums[tid] = from < (int)cluster.num_blocks()
                    ? *cluster.map_shared_rank(&mine[pass & 1][tid % kVfWarps], from)
                    : Pair{0.f, 0.f};
  }
  __syncthreads();
}

// What lies before the lane's segments and up to each of them; returns the total.
// Every warp of every CTA adds in the same order.
template <int kPer>
__device__ __forceinline__ Pair scan_sums(const Pair *sums, Pair &before, Pair (&upto)[kPer]) {
  const int lane = threadIdx.x & 31;
  upto[0] = sums[kPer * lane];
#pragma unroll
  for (int k = 1; k < kPer; ++k) upto[k] = plus(upto[k - 1], sums[kPer * lane + k]);
  before = shfl_up(warp_upto(upto[kPer - 1]), 1);
  if (lane == 0) before = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kPer; ++k) upto[k] = plus(before, upto[k]);
  return shfl(upto[kPer - 1], 31);
}

// kRanks: CTAs of a cluster, at most; kAhead: rows of both probabilities in flight,
// four with four CTAs on an SM, eight with two.
template <bool kVec, int kRanks, int kAhead>
__global__ void __launch_bounds__(kVfThreads, 16 / kAhead) verify_kernel(const VerifyParams p) {
  __shared__ int n_par[kVfNodes], n_tok[kVfNodes];
  __shared__ float n_u[kVfNodes], n_p[kVfNodes], n_q[kVfNodes];
  __shared__ Pair mine[2][kVfWarps];  // this CTA's segment sums, of alternate passes
  // segments of a lane, where a warp scans their sums
  constexpr int kPer = kRanks * kVfWarps / 32;
  static_assert(kRanks * kVfWarps <= kVfThreads, "a thread fetches each segment's sum");
  __shared__ Pair sums[kRanks * kVfWarps];  // all CTAs', of the last pass
  __shared__ Pair s_beta, s_rows[kVfWarps];
  __shared__ int s_cur, s_act, s_next, s_count, s_best[2];
  extern __shared__ uint32_t out_bits[];  // looked-up guesses rejected at this node
  cg::cluster_group cluster = cg::this_cluster();
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int seq = (int)blockIdx.x / ranks;
  const bool first = rank == 0;
  const int q0 = p.cu[seq], end = p.cu[seq + 1];
  const long long nl = (long long)end - q0;
  int32_t *path = p.path + (long long)seq * p.width;
  int32_t *toks = p.out_tokens + (long long)seq * p.width;
  const bool fits = nl == 0 || (q0 >= 0 && end <= p.total && nl > 0 && nl <= p.width);
  if (nl == 0 || !fits) {  // (the whole cluster)
    if (first) {
      if (!fits && tid == 0) report(p.err, PA_DEVERR_SHAPE);
      if (tid == 0) p.accepted[seq] = 0;
      for (int i = tid; i < p.width; i += kVfThreads) path[i] = toks[i] = -1;
    }
    return;
  }
  const int nodes = (int)nl;
  const bool looked = p.q == nullptr;
  if (looked)
    for (int i = tid; i < (p.vocab + 31) / 32; i += kVfThreads) out_bits[i] = 0u;
  const int s0 = (int)min((long long)p.vocab, (long long)(rank * kVfWarps + warp) * p.segment);
  const int s1 = min(p.vocab, s0 + p.segment);

  // The walk, by warp 0 of every CTA alike, over nodes held in shared memory,
  // until it needs more of them, the weights' sum, or no more.
  enum { kLoad, kPass, kSum, kDone };
  int cur = 0, count = 1, at = 0;  // node, nodes so far, last node looked at
  int held = 0, passes = 0;        // nodes held .. held + kVfNodes - 1 are there
  const Pair zero = {0.f, 0.f}, one = {1.f, 0.f};
  Pair beta = zero, mass = one, gone = zero;
  bool dirty = false;   // a bit of out_bits is set
  bool summed = false;  // `sums` are those of the present weights
  if (first && tid == 0) path[0] = 0;
  if (tid == 0) {
    s_act = nodes > 1 ? kLoad : kSum;
    s_next = 1;
    s_cur = 0;
    s_beta = zero;
    s_count = 1;
  }
  __syncthreads();
  while (s_act != kDone) {
    if (s_act == kLoad) {
      held = s_next;
      for (int i = tid; i < kVfNodes && held + i < nodes; i += kVfThreads) {
        const int j = held + i;
        int par = p.parents[q0 + j], tok = p.tokens[q0 + j];
        if (par >= j) {
          if (first) report(p.err, PA_DEVERR_SHAPE);
          par = -1;
        }
        if (tok < 0 || tok >= p.vocab) tok = -1;
        const bool there = par >= 0 && tok >= 0;
        n_par[i] = par;
        n_tok[i] = tok;
        n_u[i] = p.u[q0 + j];
        n_p[i] = there ? p.p[(q0 + par) * p.p_stride + tok] : 0.f;
        n_q[i] = there && !looked ? p.q[(q0 + par) * p.q_stride + tok] : 0.f;
      }
      __syncthreads();
    } else {  // kPass, kSum
      const long long row = q0 + s_cur;
      const bool plain = looked || s_beta.hi == 0.f;
      const Rows r{p.p + row * p.p_stride, plain ? nullptr : p.q + row * p.q_stride, s_beta.hi,
                   s_beta.lo};
      const bool last = s_act == kSum;
      sum_rows<kVec, kRanks, kAhead>(cluster, r, looked ? out_bits : nullptr, s0, s1, mine, sums, passes++);
      if (last) break;
    }
    if (warp == 0) {
      if (s_act == kPass) {
        Pair before, upto[kPer];
        mass = scan_sums(sums, before, upto);
        summed = true;
      }
      int act = kLoad;
      while (true) {
        if (at + 1 >= nodes) {
          act = summed ? kDone : kSum;
          break;
        }
        if (at + 1 >= held + kVfNodes) break;  // kLoad
        // the next child of cur among the 32 nodes from at + 1 on
        const int i = at + 1 - held + lane;
        const bool in = i < kVfNodes && held + i < nodes;
        const unsigned kids = __ballot_sync(0xffffffffu, in && n_par[i] == cur);
        if (!kids) {
          at = min(at + 32, min(nodes, held + kVfNodes) - 1);
          continue;
        }
        const int j = at + __ffs(kids) - held;  // its place
        at = held + j;
        const int tok = n_tok[j];
        if (tok < 0) {
          if (first && lane == 0) report(p.err, PA_DEVERR_TOKEN);
          continue;
        }
        bool ok;
        if (looked) {
          const bool was = (out_bits[tok >> 5] >> (tok & 31)) & 1u;
          const Pair px = {was ? 0.f : n_p[j], 0.f};
          ok = above(px, times({n_u[j], 0.f}, mass));
          if (!ok) {
            if (px.hi > 0.f) mass = minus(mass, px);
            if (!(mass.hi > 0.f)) mass = zero;
            __syncwarp();
            if (lane == 0) out_bits[tok >> 5] |= 1u << (tok & 31);
            __syncwarp();
            dirty = true;
          }
        } else {
          // (the first child of a node: u q < p, exact)
          const bool sole = gone.hi == 0.f;
          Pair left = one;
          if (!sole) left = minus(one, gone);
          if (left.hi < kVfLeast) left = {kVfLeast, 0.f};
          const Pair qx = {n_q[j], 0.f};
          Pair rest = {n_p[j], 0.f}, draw = times({n_u[j], 0.f}, qx);
          if (beta.hi != 0.f) {
            rest = minus(rest, times(beta, qx));
            draw = times(draw, mass);
            if (!sole) rest = times(rest, left);
          }
          ok = above(rest, draw);
          if (!ok) {
            beta = plus(beta, sole ? mass : over(mass, left));
            if (!p.again) gone = plus(gone, qx);
            act = kPass;
            break;
          }
        }
        if (ok) {
          if (first && lane == 0) {
            path[count] = at;
            toks[count - 1] = tok;
          }
          ++count;
          cur = at;
          beta = gone = zero;
          mass = one;
          summed = false;
          if (dirty) {
            for (int i = lane; i < (p.vocab + 31) / 32; i += 32) out_bits[i] = 0u;
            __syncwarp();
            dirty = false;
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        s_act = act;
        s_next = at + 1;
        s_cur = cur;
        s_beta = beta;
        s_count = count;
      }
    }
    __syncthreads();
  }

  // The token after: its segment by the sums, then the segment alone.
  count = s_count;
  const long long row = q0 + s_cur;
  Rows r{p.p + row * p.p_stride, looked || s_beta.hi == 0.f ? nullptr : p.q + row * p.q_stride,
         s_beta.hi, s_beta.lo};
  const uint32_t *out = looked ? out_bits : nullptr;
  Pair before, upto[kPer], total = scan_sums(sums, before, upto);
  if (!(total.hi > 0.f)) {  // nothing left, by rounding alone: the target's row
    __syncthreads();        // all warps have read `sums`
    r.q = nullptr;
    out = nullptr;
    sum_rows<kVec, kRanks, kAhead>(cluster, r, out, s0, s1, mine, sums, passes++);
    total = scan_sums(sums, before, upto);
  }
  const float ul = p.u_last[seq], th = ul * total.hi;  // u' times the total
  const float tl = fmaf(ul, total.hi, -th) + ul * total.lo, t2 = th + tl;
  const Pair target = {t2, tl - (t2 - th)};
  int seg = INT_MAX, filled = -1;
#pragma unroll
  for (int k = kPer - 1; k >= 0; --k) {
    if (sums[kPer * lane + k].hi > 0.f) {
      filled = max(filled, kPer * lane + k);
      if (above(upto[k], target)) seg = kPer * lane + k;
    }
  }
  seg = __reduce_min_sync(0xffffffffu, seg);
  filled = __reduce_max_sync(0xffffffffu, filled);
  if (seg == INT_MAX) seg = filled;  // -1: no weight at all
  if (seg >= 0 && seg / kVfWarps == rank) {  // (the whole CTA)
    Pair at0 = before;
#pragma unroll
    for (int k = 1; k < kPer; ++k)
      if (seg % kPer == k) at0 = upto[k - 1];
    at0 = shfl(at0, seg / kPer);
    const int f0 = seg * p.segment, f1 = min(p.vocab, f0 + p.segment);
    const int tok = segment_find<kVec>(r, f0, f1, out, at0, target, s_rows, s_best);
    if (tid == 0) toks[count - 1] = tok;
  }
  if (first) {
    if (tid == 0) {
      p.accepted[seq] = count;
      if (seg < 0) toks[count - 1] = -1;
    }
    for (int i = count + tid; i < p.width; i += kVfThreads) path[i] = toks[i] = -1;
  }
  cluster.sync();  // no CTA leaves while another reads its sums
}

// CTAs of a sequence's cluster: more while every warp then has a row of 128 tokens
// and all clusters run at once, four CTAs per SM; sixteen (more than is portable)
// only where a warp still has four rows.  Measured, us: 64 sequences at 151936
// tokens, 8 CTAs of 256 threads 35 (4 of 512 40, 8 of 512 64, 16 of 128 36); 16 at
// 128000, 16 CTAs 19.5, 8 23.2; one at 32000, 8 CTAs 6.3, 16 7.0; 256 at 32000, 2 CTAs
// 27.5, one of 512 threads 31, 8 of 512 93.
constexpr int kVfRanks = 8, kVfMoreRanks = 16;
int verify_ranks(int vocab, int seqs, int sms) {
  int ranks = 1;
  while (ranks < kVfRanks && vocab > ranks * kVfWarps * 128 && ranks * (long long)seqs <= 2 * sms)
    ranks *= 2;
  if (ranks == kVfRanks && vocab >= kVfMoreRanks * kVfWarps * 512 &&
      kVfMoreRanks * (long long)seqs <= 4 * sms)
    ranks = kVfMoreRanks;
  return ranks;
}

template <bool kVec, int kRanks, int kAhead>
cudaError_t launch_verify(const VerifyParams &p, int ranks, size_t bits, int device,
                          cudaStream_t s) {
  static std::atomic<bool> configured[64] = {};
  auto kernel = verify_kernel<kVec, kRanks, kAhead>;
  cudaError_t e = set_smem_once(configured, kernel, device, kVfMaxVocab / 8);
  if (e == cudaSuccess && kRanks > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, dim3((unsigned)(p.num_seqs * ranks)), dim3(kVfThreads),
                        (unsigned)ranks, bits, s, p);
}
// Clusters of sixteen CTAs, two per SM, that the device runs at once (a cluster stays
// within a part of the chip, so fewer than its SMs would hold); asked once.
template <bool kVec>
int wide_clusters(int device) {
  static std::atomic<int> known[64] = {};
  const bool tracked = device >= 0 && device < 64;
  int n = tracked ? known[device].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n - 1;
  auto kernel = verify_kernel<kVec, kVfMoreRanks, 8>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kVfMoreRanks);
  cfg.blockDim = dim3(kVfThreads);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kVfMoreRanks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (tracked) known[device].store(n + 1, std::memory_order_relaxed);
  return n;
}
template <bool kVec>
cudaError_t launch_verify(const VerifyParams &p, int ranks, size_t bits, int device,
                          cudaStream_t s) {
  if (ranks <= kVfRanks) return launch_verify<kVec, kVfRanks, 4>(p, ranks, bits, device, s);
  return p.num_seqs <= wide_clusters<kVec>(device)
             ? launch_verify<kVec, kVfMoreRanks, 8>(p, ranks, bits, device, s)
             : launch_verify<kVec, kVfMoreRanks, 4>(p, ranks, bits, device, s);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_verify_tree(int32_t *accepted, int32_t *path, int32_t *out_tokens,
                                    const int32_t *tokens, const int32_t *parents,
                                    const int32_t *cu_seqlens, int32_t num_seqs,
                                    int32_t total_tokens, int32_t max_q_len,
                                    const float *target_probs, int64_t target_stride,
                                    const float *draft_probs, int64_t draft_stride,
                                    int32_t vocab_size, const float *uniforms,
                                    const float *sample_uniforms, int32_t draws,
                                    int32_t *error_flags, uint32_t flags, void *stream) {
  using namespace pa;
  if (num_seqs < 0 || total_tokens < 0 || max_q_len < 0 || vocab_size < 0) return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (draws != PA_DRAWS_WITHOUT_REPLACEMENT && draws != PA_DRAWS_WITH_REPLACEMENT)
    return PA_ERR_INVALID_ARG;
  if (vocab_size > kVfMaxVocab) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (num_seqs > INT_MAX / kVfMoreRanks) return PA_ERR_UNSUPPORTED;
  if (!accepted || !cu_seqlens || !sample_uniforms) return PA_ERR_INVALID_ARG;
  if (max_q_len > 0 && (!path || !out_tokens)) return PA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!tokens || !parents || !target_probs || !uniforms || vocab_size < 1))
    return PA_ERR_INVALID_ARG;
  if (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size))
    return PA_ERR_INVALID_ARG;
  for (const void *x : {(const void *)accepted, (const void *)path, (const void *)out_tokens,
                        (const void *)tokens, (const void *)parents, (const void *)cu_seqlens,
                        (const void *)target_probs, (const void *)draft_probs,
                        (const void *)uniforms, (const void *)sample_uniforms,
                        (const void *)error_flags})
    if (reinterpret_cast<uintptr_t>(x) & 3) return PA_ERR_INVALID_ARG;
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_DEVICE;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return PA_ERR_DEVICE;
  const int ranks = verify_ranks(vocab_size, num_seqs, sms);
  VerifyParams p;
  p.accepted = accepted;
  p.path = path;
  p.out_tokens = out_tokens;
  p.tokens = tokens;
  p.parents = parents;
  p.cu = cu_seqlens;
  p.num_seqs = num_seqs;
  p.total = total_tokens;
  p.width = max_q_len;
  p.p = target_probs;
  p.p_stride = target_stride;
  p.q = draft_probs;
  p.q_stride = draft_stride;
  p.vocab = vocab_size;
  p.u = uniforms;
  p.u_last = sample_uniforms;
  p.again = draws == PA_DRAWS_WITH_REPLACEMENT;
  const int per = (vocab_size + ranks * kVfWarps - 1) / (ranks * kVfWarps);
  p.segment = (per + 127) / 128 * 128;
  p.err = error_flags;
  const bool vec = ((reinterpret_cast<uintptr_t>(target_probs) |
                     reinterpret_cast<uintptr_t>(draft_probs)) % 16 == 0) &&
                   target_stride % 4 == 0 && (!draft_probs || draft_stride % 4 == 0);
  const size_t bits = draft_probs ? 0 : (size_t)(vocab_size + 31) / 32 * 4;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = vec ? launch_verify<true>(p, ranks, bits, device, st)
                            : launch_verify<false>(p, ranks, bits, device, st);
  if (e != cudaSuccess) return PA_ERR_LAUNCH;
  return PA_OK;
}
