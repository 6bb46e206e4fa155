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
// element.  fp64 is for the tests of single nodes alone: its rate on this chip is
// so low that joining lanes and segments in it took 61 us for 64 sequences of
// 32000 tokens against 12 for one.
//
// Bound by latency for few sequences, and by HBM for many: a pass reads 8 bytes
// an element.
#include <climits>

#include <cooperative_groups.h>

#include "pa_common.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kVfThreads = 512, kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 8;
constexpr int kVfSegments = kVfMaxCluster * kVfWarps;
constexpr int kVfNodes = 256;          // nodes whose elements are held at a time
constexpr int kVfMaxVocab = 1 << 20;   // (a bit for each token, in shared memory)
constexpr double kVfLeast = 1.0 / (1 << 24);

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
  const float ph = q * bh;
  const float pl = fmaf(q, bl, fmaf(q, bh, -ph));
  const float s = p - ph, bb = s - p;
  const float lo = ((p - (s - bb)) - (ph + bb)) - pl;  // p - ph = s + ...
  const float hi = s + lo;
  return {hi > 0.f ? hi : 0.f, hi > 0.f ? lo - (hi - s) : 0.f};
}
// a + x without bringing hi up to date: x's low part and the error go to lo.
__device__ __forceinline__ void add(Pair &a, const Pair &x) {
  const float s = a.hi + x.hi, bb = s - a.hi;
  a.lo += ((a.hi - (s - bb)) + (x.hi - bb)) + x.lo;
  a.hi = s;
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
template <bool kVec>
__device__ Pair segment_sum(const Rows &r, int s0, int s1, const uint32_t *out) {
  const int lane = threadIdx.x & 31;
  Pair acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
  constexpr int kAhead = 4;
  for (int i0 = s0 + 4 * lane; i0 - 4 * lane < s1; i0 += 128 * kAhead) {
    float p[kAhead][4], q[kAhead][4];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + 128 * a;
      load4<kVec>(r.p, i, s1 - i, p[a]);
      if (r.q) load4<kVec>(r.q, i, s1 - i, q[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      Pair w[4];
      if (i0 + 128 * a < s1) {
        weights4(r, p[a], q[a], out, i0 + 128 * a, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) add(acc[k], w[k]);
      }
    }
  }
  Pair sum = plus(plus(acc[0], acc[1]), plus(acc[2], acc[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    sum = plus(sum, {__shfl_xor_sync(0xffffffffu, sum.hi, o),
                     __shfl_xor_sync(0xffffffffu, sum.lo, o)});
  return sum;
}

// The first token of segment [s0, s1) where `before` plus the running sum is over
// `target`; its last of positive weight if there is none (-1: no such).
template <bool kVec>
__device__ int segment_find(const Rows &r, int s0, int s1, const uint32_t *out, Pair before,
                            const Pair &target) {
  const int lane = threadIdx.x & 31;
  int last = -1;
  constexpr int kAhead = 2;
  for (int b = s0; b < s1; b += 128 * kAhead) {
    float p[kAhead][4], q[kAhead][4];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = b + 128 * a + 4 * lane;
      load4<kVec>(r.p, i, s1 - i, p[a]);
      if (r.q) load4<kVec>(r.q, i, s1 - i, q[a]);
    }
    Pair upto[kAhead], c[kAhead][4];
    int mine = -1;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = b + 128 * a + 4 * lane;
      Pair w[4];
      weights4(r, p[a], q[a], out, i, w);
      c[a][0] = w[0];
#pragma unroll
      for (int k = 1; k < 4; ++k) c[a][k] = plus(c[a][k - 1], w[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (w[k].hi > 0.f)
          mine = i + k;
        else
          c[a][k].hi = -1.f;  // (no token to draw: below any target)
      }
      Pair run = plus(plus(w[0], w[1]), plus(w[2], w[3]));
      upto[a] = warp_upto(run);
    }
    int found = INT_MAX;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      Pair base = shfl_up(upto[a], 1);
      base = lane == 0 ? before : plus(before, base);
#pragma unroll
      for (int k = 3; k >= 0; --k)
        if (c[a][k].hi > 0.f && above(plus(base, c[a][k]), target))
          found = min(found, b + 128 * a + 4 * lane + k);
      before = plus(before, shfl(upto[a], 31));
    }
    found = __reduce_min_sync(0xffffffffu, found);
    if (found != INT_MAX) return found;
    last = max(last, __reduce_max_sync(0xffffffffu, mine));
  }
  return last;
}

// All segments' sums into `sums` of every CTA of the cluster.  Alternate passes use
// alternate halves of `mine`: a CTA still reads one pass's while another writes the
// next one's, and the pass after that waits for it at the barrier between.
template <bool kVec>
__device__ void sum_rows(cg::cluster_group &cluster, const Rows &r, const uint32_t *out, int s0,
                         int s1, Pair (&mine)[2][kVfWarps], Pair *sums, int pass) {
  const int tid = threadIdx.x, warp = tid >> 5;
  const Pair sum = segment_sum<kVec>(r, s0, s1, out);
  if ((tid & 31) == 0) mine[pass & 1][warp] = sum;
  cluster.sync();
  if (tid < kVfSegments) {
    const int from = tid / kVfWarps;
    sums[tid] = from < (int)cluster.num_blocks()
                    ? *cluster.map_shared_rank(&mine[pass & 1][tid % kVfWarps], from)
                    : Pair{0.f, 0.f};
  }
  __syncthreads();
}

// What lies before the lane's four segments and up to each of them; returns the
// total.  Every warp of every CTA adds in the same order.
__device__ __forceinline__ Pair scan_sums(const Pair *sums, Pair &before, Pair (&upto)[4]) {
  static_assert(kVfSegments == 128, "four segments a lane");
  const int lane = threadIdx.x & 31;
  upto[0] = sums[4 * lane];
#pragma unroll
  for (int k = 1; k < 4; ++k) upto[k] = plus(upto[k - 1], sums[4 * lane + k]);
  before = shfl_up(warp_upto(upto[3]), 1);
  if (lane == 0) before = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k) upto[k] = plus(before, upto[k]);
  return shfl(upto[3], 31);
}

template <bool kVec>
__global__ void __launch_bounds__(kVfThreads, 2) verify_kernel(const VerifyParams p) {
  __shared__ int n_par[kVfNodes], n_tok[kVfNodes];
  __shared__ float n_u[kVfNodes], n_p[kVfNodes], n_q[kVfNodes];
  __shared__ Pair mine[2][kVfWarps];  // this CTA's segment sums, of alternate passes
  __shared__ Pair sums[kVfSegments];  // all CTAs', of the last pass
  __shared__ double s_beta;
  __shared__ int s_cur, s_act, s_next, s_count;
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
  double beta = 0.0, mass = 1.0, gone = 0.0;
  bool dirty = false;   // a bit of out_bits is set
  bool summed = false;  // `sums` are those of the present weights
  if (first && tid == 0) path[0] = 0;
  if (tid == 0) {
    s_act = nodes > 1 ? kLoad : kSum;
    s_next = 1;
    s_cur = 0;
    s_beta = 0.0;
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
      const float bh = (float)s_beta, bl = (float)(s_beta - (double)bh);
      const long long row = q0 + s_cur;
      const bool plain = looked || s_beta == 0.0;
      const Rows r{p.p + row * p.p_stride, plain ? nullptr : p.q + row * p.q_stride, bh, bl};
      const bool last = s_act == kSum;
      sum_rows<kVec>(cluster, r, looked ? out_bits : nullptr, s0, s1, mine, sums, passes++);
      if (last) break;
    }
    if (warp == 0) {
      if (s_act == kPass) {
        Pair before, upto[4];
        const Pair total = scan_sums(sums, before, upto);
        mass = (double)total.hi + (double)total.lo;
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
          const double px = was ? 0.0 : (double)n_p[j];
          ok = (double)n_u[j] * mass < px;
          if (!ok) {
            if (px > 0.0) mass = fmax(mass - px, 0.0);
            __syncwarp();
            if (lane == 0) out_bits[tok >> 5] |= 1u << (tok & 31);
            __syncwarp();
            dirty = true;
          }
        } else {
          // (the first child of a node: u q < p, exact)
          const double left = gone == 0.0 ? 1.0 : fmax(1.0 - gone, kVfLeast);
          const double qx = (double)n_q[j];
          ok = (double)n_u[j] * qx * mass < left * fma(-beta, qx, (double)n_p[j]);
          if (!ok) {
            beta += gone == 0.0 ? mass : mass / left;
            if (!p.again) gone += qx;
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
          beta = gone = 0.0;
          mass = 1.0;
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
  const float bh = (float)s_beta, bl = (float)(s_beta - (double)bh);
  Rows r{p.p + row * p.p_stride, looked || s_beta == 0.0 ? nullptr : p.q + row * p.q_stride, bh,
         bl};
  const uint32_t *out = looked ? out_bits : nullptr;
  Pair before, upto[4], total = scan_sums(sums, before, upto);
  if (!(total.hi > 0.f)) {  // nothing left, by rounding alone: the target's row
    __syncthreads();        // all warps have read `sums`
    r.q = nullptr;
    out = nullptr;
    sum_rows<kVec>(cluster, r, out, s0, s1, mine, sums, passes++);
    total = scan_sums(sums, before, upto);
  }
  const float ul = p.u_last[seq], th = ul * total.hi;  // u' times the total
  const float tl = fmaf(ul, total.hi, -th) + ul * total.lo, t2 = th + tl;
  const Pair target = {t2, tl - (t2 - th)};
  int seg = INT_MAX, filled = -1;
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    if (sums[4 * lane + k].hi > 0.f) {
      filled = max(filled, 4 * lane + k);
      if (above(upto[k], target)) seg = 4 * lane + k;
    }
  }
  seg = __reduce_min_sync(0xffffffffu, seg);
  filled = __reduce_max_sync(0xffffffffu, filled);
  if (seg == INT_MAX) seg = filled;  // -1: no weight at all
  if (seg == rank * kVfWarps + warp) {
    const int k = seg & 3;
    const Pair at0 = shfl(k == 0 ? before : k == 1 ? upto[0] : k == 2 ? upto[1] : upto[2],
                          seg >> 2);
    const int tok = segment_find<kVec>(r, s0, s1, out, at0, target);
    if (lane == 0) toks[count - 1] = tok;
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

// CTAs of a cluster, for a vocabulary: a warp has 128 tokens at a time, and none
// without any.
int verify_ranks(int vocab) {
  int ranks = 1;
  while (ranks < kVfMaxCluster && vocab > ranks * kVfWarps * 128) ranks *= 2;
  return ranks;
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
  if (num_seqs > INT_MAX / kVfMaxCluster) return PA_ERR_UNSUPPORTED;
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
  const int ranks = verify_ranks(vocab_size);
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
  constexpr int kMostBits = kVfMaxVocab / 8;
  static std::atomic<bool> set_vec[64] = {}, set_any[64] = {};
  const cudaError_t e = vec ? set_smem_once(set_vec, verify_kernel<true>, device, kMostBits)
                            : set_smem_once(set_any, verify_kernel<false>, device, kMostBits);
  if (e != cudaSuccess) return PA_ERR_LAUNCH;
  if (launch_cluster(vec ? verify_kernel<true> : verify_kernel<false>,
                     dim3((unsigned)(num_seqs * ranks)), dim3(kVfThreads), (unsigned)ranks, bits,
                     static_cast<cudaStream_t>(stream), p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}
