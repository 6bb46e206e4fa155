// Page operators over a block-paged cache whose pages are shared by reference
// counts: copy (pa_copy_pages), fork (pa_fork_pages), free (pa_free_pages) and
// compact (pa_compact_pages).  A page's count is the number of table entries
// that name it; count 0 is a free page.  The counts alone are the allocator's
// state: a fork takes the lowest free pages, so results do not depend on the
// order in which blocks of a launch run (the counts are integer sums).
//
// Every kernel here is launched as a programmatic dependent, waits for the
// kernel before it first of all and reads with plain loads (that kernel may
// have written anything while this one was set up), so that only its set-up
// moves ahead, about 2 us of a call behind another.
//
// Fork and compact are planned by one block, since every pick depends on all
// earlier ones (a scan over the counts); a second launch, spread over the
// sequences, applies the plan.  Nothing is read back to the host: the plan's
// page pairs go to pa_copy_pages through device memory.
#include <climits>

#include "pa_common.cuh"

namespace pa {
namespace {

// ---- copy ---------------------------------------------------------------------
// out[p][dst[i]] = out[p][src[i]] for every pool p and pair i.  Bound by HBM:
// each byte is read and written once.  The work of a pair is the list of all
// pools' pages cut into 4 KB chunks; a warp moves a chunk with eight 16-byte
// loads per lane in flight.  Pages of up to 16 bytes (scale bytes) would
// waste a warp each: 32 of them make one unit, a lane each.
constexpr int kCopyPools = 128;  // pools per launch
constexpr int kCopyChunk = 4096;
constexpr int kCopyWarps = 8;

struct CopyPool {
  uint8_t *base;
  long long page_bytes;
};
struct CopyPagesParams {
  CopyPool pool[kCopyPools];
  int chunk_end[kCopyPools];  // chunks of pools 0 .. p of one pair
  int vec[kCopyPools / 32];   // bit p: 16-byte chunks
  int num_big, num_tiny;      // pools [0, num_big) in chunks, the next num_tiny by lanes
  long long num_blocks;
  const int32_t *src, *dst;
  int num_pairs;
  const int32_t *count;
  int32_t *err;
};

__global__ void __launch_bounds__(32 * kCopyWarps) copy_pages_kernel(
    const __grid_constant__ CopyPagesParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  int pairs = p.num_pairs;
  if (p.count) pairs = min(pairs, max(*p.count, 0));
  const int per = p.num_big ? p.chunk_end[p.num_big - 1] : 0;
  const long long big = (long long)pairs * per, tiny = (long long)pairs * p.num_tiny;
  const long long units = big + (tiny + 31) / 32;
  const long long stride = (long long)gridDim.x * kCopyWarps;
  for (long long u = (long long)blockIdx.x * kCopyWarps + (threadIdx.x >> 5); u < units;
       u += stride) {
    if (u >= big) {  // tiny pages, a lane each
      const long long t = (u - big) * 32 + lane;
      if (t >= tiny) continue;
      const int i = (int)(t / p.num_tiny), q = p.num_big + (int)(t % p.num_tiny);
      const long long s = p.src[i], d = p.dst[i];
      if (s < 0) continue;
      if (s >= p.num_blocks || d < 0 || d >= p.num_blocks) {
        report(p.err, PA_DEVERR_BLOCK_INDEX);
        continue;
      }
      const int n = (int)p.pool[q].page_bytes;
      const uint8_t *from = p.pool[q].base + s * n;
      uint8_t *to = p.pool[q].base + d * n;
      for (int k = 0; k < n; ++k) to[k] = from[k];
      continue;
    }
    const int i = (int)(u / per), c = (int)(u % per);
    const long long s = p.src[i], d = p.dst[i];
    if (s < 0) continue;
    if (s >= p.num_blocks || d < 0 || d >= p.num_blocks) {
      if (c == 0 && lane == 0) report(p.err, PA_DEVERR_BLOCK_INDEX);
      continue;
    }
    int lo = 0, hi = p.num_big - 1;  // the pool of chunk c
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (c < p.chunk_end[mid])
        hi = mid;
      else
        lo = mid + 1;
    }
    const long long bytes = p.pool[lo].page_bytes;
    const long long off = (long long)(c - (lo ? p.chunk_end[lo - 1] : 0)) * kCopyChunk;
    const int n = (int)min((long long)kCopyChunk, bytes - off);
    const uint8_t *from = p.pool[lo].base + s * bytes + off;
    uint8_t *to = p.pool[lo].base + d * bytes + off;
    if ((p.vec[lo >> 5] >> (lo & 31)) & 1) {
      uint4 v[kCopyChunk / 512];
#pragma unroll
      for (int k = 0; k < kCopyChunk / 512; ++k)
        if (512 * k + 16 * lane < n) v[k] = *reinterpret_cast<const uint4 *>(from + 512 * k + 16 * lane);
#pragma unroll
      for (int k = 0; k < kCopyChunk / 512; ++k)
        if (512 * k + 16 * lane < n) *reinterpret_cast<uint4 *>(to + 512 * k + 16 * lane) = v[k];
    } else {
      for (int k = lane; k < n; k += 32) to[k] = from[k];
    }
  }
}

// ---- plans: one block -----------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 8;  // pages a thread looks at in one step
// A fork of at most this many table entries (rows at their full width) is
// applied by the plan's own block, a launch less; beyond, spread over the SMs.
constexpr long long kInlineEntries = 4096;

// Exclusive sum over the block's threads of v, and the total.
__device__ __forceinline__ int plan_scan(int v, int *wsum, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  int w = wsum[lane];  // 32 warps
  int incl = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  total = __shfl_sync(0xffffffffu, incl, 31);
  const int before = __shfl_sync(0xffffffffu, incl - w, warp);
  __syncthreads();  // wsum is reused by the next scan
  return before + x - v;
}

// Bit k: page first + k has a count of 0 (pages past the pool: not set).
__device__ __forceinline__ unsigned free_mask(const int32_t *refs, long long first,
                                              long long num_blocks) {
  unsigned m = 0;
  if (first + kPlanPer <= num_blocks && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
    const int4 a = *reinterpret_cast<const int4 *>(refs + first);
    const int4 b = *reinterpret_cast<const int4 *>(refs + first + 4);
    const int v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) m |= (v[k] <= 0 ? 1u : 0u) << k;
  } else {
    for (int k = 0; k < kPlanPer; ++k)
      if (first + k < num_blocks && refs[first + k] <= 0) m |= 1u << k;
  }
  return m;
}

struct ForkParams {
  int32_t *tables;
  long long stride;
  int32_t *ctx;
  int rows;
  const int32_t *parents, *children;
  int n;
  int32_t *refs;
  long long num_blocks;
  int32_t *src, *dst, *forked;
  int32_t *err;
  int apply;  // the plan's block applies it too
};

// A fork's plan: rows, the child's length (-1: refused), the page to copy
// (-1: none) and its copy.
struct Fork {
  int parent, child, n, src, dst;
};

// The fork's table row: the child's entries j0, j0 + step, ...
__device__ __forceinline__ void apply_fork(const ForkParams &p, const Fork &f, int j0, int step) {
  const int n = f.n;
  if (n < 0) return;
  const int k = ceil_div_blocks(n);
  const int last = f.src >= 0 ? k - 1 : -1;
  const int32_t *from = p.tables + (long long)f.parent * p.stride;
  int32_t *to = p.tables + (long long)f.child * p.stride;
  for (int j = j0; j < k; j += step) {
    const int page = j == last ? f.dst : from[j];
    to[j] = page;
    if (page >= 0 && page < p.num_blocks)
      atomicAdd(p.refs + page, 1);
    else
      report(p.err, PA_DEVERR_BLOCK_INDEX);
  }
  if (j0 == 0) p.ctx[f.child] = n;
}

// Fork i is refused when its parent or child is no row, they are the same,
// the child holds pages or is an earlier fork's child, or the parent's
// context does not fit its table row.  The children claim their rows: the
// context length of an empty child row takes INT_MIN + i of the lowest fork i
// that names it until the plan is applied (a length below 1 reads as empty; a
// negative one becomes 0 first, so that none is taken for a claim).
//
// The plan is a chain of dependent loads by one block (about 4 us), so up to
// 1024 forks keep their rows and plan in shared memory between its steps.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int wsum[32];
  __shared__ int kept[5][kPlanThreads];
  const int tid = threadIdx.x;
  volatile int32_t *ctx = p.ctx;
  const bool small = p.n <= kPlanThreads;
  const int32_t *parents = small ? kept[0] : p.parents, *children = small ? kept[1] : p.children;
  int32_t *src = small ? kept[2] : p.src, *dst = small ? kept[3] : p.dst;
  int32_t *forked = small ? kept[4] : p.forked;
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int c = p.children[i];
    if (small) {
      kept[0][i] = p.parents[i];
      kept[1][i] = c;
    }
    if (c >= 0 && c < p.rows && ctx[c] < 0) ctx[c] = 0;
  }
  // the first pages' counts, for step 3
  unsigned first_mask = 0;
  if ((long long)tid * kPlanPer < p.num_blocks)
    first_mask = free_mask(p.refs, (long long)tid * kPlanPer, p.num_blocks);
  __syncthreads();
  auto length = [&](int i) {  // the parent's context length; -1: refused
    const int a = parents[i], c = children[i];
    if (a < 0 || a >= p.rows || c < 0 || c >= p.rows || a == c) return -1;
    const int n = ctx[a];
    if (n > 0 && (long long)(n - 1) / kBlockSize >= p.stride) return -1;
    return max(n, 0);
  };
  // 1. claims
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int n = length(i);
    if (n >= 0 && ctx[children[i]] <= 0) atomicMin(p.ctx + children[i], INT_MIN + i);
  }
  __syncthreads();
  // 2. ranks of the forks that need a page of their own; src[r] = fork of rank r
  int need = 0;
  for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int want = 0;
    if (i < p.n) {
      const int n = length(i);
      const bool ok = n >= 0 && ctx[children[i]] == INT_MIN + i;
      forked[i] = ok ? n : -1;
      dst[i] = -1;
      if (!ok) report(p.err, PA_DEVERR_SHAPE);
      want = ok && n % kBlockSize != 0;
    }
    int total;
    const int r = need + plan_scan(want, wsum, total);
    if (want) src[r] = i;
    need += total;
  }
  __syncthreads();
  // 3. the lowest free pages, in order
  int found = 0;
  for (long long b = 0; b < p.num_blocks && found < need; b += kPlanThreads * kPlanPer) {
    const long long first = b + (long long)tid * kPlanPer;
    unsigned m = b == 0 ? first_mask
                        : first < p.num_blocks ? free_mask(p.refs, first, p.num_blocks) : 0u;
    int total;
    int r = found + plan_scan(__popc(m), wsum, total);
    for (; m && r < need; m &= m - 1, ++r) dst[src[r]] = (int)(first + __ffs(m) - 1);
    found += total;
  }
  __syncthreads();
  // 4. the pairs
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int n = forked[i], c = children[i];
    int s = -1;
    if (n > 0 && n % kBlockSize != 0) {
      if (dst[i] >= 0) {
        s = p.tables[(long long)parents[i] * p.stride + n / kBlockSize];
        // an entry outside the pool is copied like any other (and reported by
        // apply_fork): the page picked for it stays free
        if (s < 0 || s >= p.num_blocks) s = dst[i] = -1;
      } else {
        forked[i] = -1;  // no page left
        report(p.err, PA_DEVERR_PAGES);
      }
    }
    // a claim that comes to nothing is given back
    if (forked[i] < 0 && c >= 0 && c < p.rows && ctx[c] == INT_MIN + i) p.ctx[c] = 0;
    src[i] = s;
    if (small) {
      p.src[i] = s;
      p.dst[i] = dst[i];
      p.forked[i] = forked[i];
    }
  }
  if (!p.apply) return;
  __syncthreads();
  // 5. few entries: a warp per fork applies it here
  for (int i = tid >> 5; i < p.n; i += kPlanThreads / 32)
    apply_fork(p, Fork{parents[i], children[i], forked[i], src[i], dst[i]}, tid & 31, 32);
}

// Block (i, y): entries of fork i's table row.
__global__ void __launch_bounds__(256) fork_apply_kernel(const ForkParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  apply_fork(p, Fork{p.parents[i], p.children[i], p.forked[i], p.src[i], p.dst[i]},
             blockIdx.y * 256 + threadIdx.x, gridDim.y * 256);
}

// ---- free: one block per row ------------------------------------------------------
__global__ void __launch_bounds__(256) free_pages_kernel(int32_t *tables, long long stride,
                                                         int32_t *ctx, int rows,
                                                         const int32_t *seqs, int32_t *refs,
                                                         long long num_blocks, int32_t *err) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int len;
  const int row = seqs[blockIdx.x];
  if (row < 0 || row >= rows) {
    if (threadIdx.x == 0) report(err, PA_DEVERR_SHAPE);
    return;
  }
  // a row named twice is freed once
  if (threadIdx.x == 0) len = atomicExch(ctx + row, 0);
  __syncthreads();
  const int n = len;
  if (n <= 0) return;
  const long long k = min((long long)ceil_div_blocks(n), stride);
  if (threadIdx.x == 0 && ceil_div_blocks(n) > stride) report(err, PA_DEVERR_SHAPE);
  for (long long j = threadIdx.x; j < k; j += blockDim.x) {
    const int page = tables[row * stride + j];
    if (page < 0 || page >= num_blocks) {
      report(err, PA_DEVERR_BLOCK_INDEX);
    } else if (atomicSub(refs + page, 1) <= 0) {
      atomicAdd(refs + page, 1);  // held by no one: the count stays
      report(err, PA_DEVERR_PAGES);
    }
  }
}

// ---- compact ------------------------------------------------------------------------
struct CompactParams {
  int32_t *tables;
  long long stride;
  const int32_t *ctx;
  int rows;
  int32_t *refs;
  long long num_blocks;
  int32_t *src, *dst, *counts, *remap;
  int32_t *err;
};

// Exclusive sums, in place, of the 256 ints of `a` by one warp; returns the total.
__device__ __forceinline__ int scan256(int *a, int lane) {
  int v[8], sum = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = a[8 * lane + k];
    sum += v[k];
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  int at = x - sum;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    a[8 * lane + k] = at;
    at += v[k];
  }
  return __shfl_sync(0xffffffffu, x, 31);
}

// With L live pages, the k-th live page at or past L (ascending) moves to the
// k-th free page before L; both lists have the same length.  Every hole comes
// before every mover in page order, so one ascending walk can pair them: a
// step (8192 pages, eight per thread, 1024 apart so that all its accesses are
// contiguous) writes its holes, and behind a barrier every hole that its
// movers need stands in dst.  Ranks are ballots within a warp over a scan of
// the step's 256 warp counts.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  static_assert(kPlanThreads == 1024 && kPlanPer == 8, "256 warp counts a step");
  __shared__ int wsum[32], hole_at[256], mover_at[256], totals[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned before = (1u << lane) - 1u;
  int mine = 0;
#pragma unroll 8
  for (long long page = tid; page < p.num_blocks; page += kPlanThreads) mine += p.refs[page] > 0;
  int live;
  plan_scan(mine, wsum, live);
  int holes = 0, movers = 0;
  for (long long b = 0; b < p.num_blocks; b += kPlanThreads * kPlanPer) {
    int ref[kPlanPer];
    unsigned hole[kPlanPer], mover[kPlanPer];
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const long long page = b + k * kPlanThreads + tid;
      ref[k] = page < p.num_blocks ? p.refs[page] : 0;
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const long long page = b + k * kPlanThreads + tid;
      hole[k] = __ballot_sync(0xffffffffu, ref[k] <= 0 && page < live);
      mover[k] = __ballot_sync(0xffffffffu, ref[k] > 0 && page >= live);
      if (lane == k) {
        hole_at[k * 32 + warp] = __popc(hole[k]);
        mover_at[k * 32 + warp] = __popc(mover[k]);
      }
    }
    __syncthreads();
    if (warp < 2) {
      const int total = scan256(warp ? mover_at : hole_at, lane);
      if (lane == 0) totals[warp] = total;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k)
      if ((hole[k] >> lane) & 1u)
        p.dst[holes + hole_at[k * 32 + warp] + __popc(hole[k] & before)] =
            (int)(b + k * kPlanThreads + tid);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const long long page = b + k * kPlanThreads + tid;
      if (page >= p.num_blocks) continue;
      int to = (int)page;
      if ((mover[k] >> lane) & 1u) {
        const int r = movers + mover_at[k * 32 + warp] + __popc(mover[k] & before);
        to = p.dst[r];
        p.src[r] = (int)page;
        p.refs[to] = ref[k];
        p.refs[page] = 0;
      }
      p.remap[page] = to;
    }
    holes += totals[0];
    movers += totals[1];
    __syncthreads();  // the counts are the next step's
  }
  if (tid == 0) {
    p.counts[0] = movers;
    p.counts[1] = live;
  }
}

// Blocks along the table rows, which also fill the lists past the moves.
__global__ void __launch_bounds__(256) compact_apply_kernel(const CompactParams p, int per_row) {
  griddep_wait();
  griddep_launch_dependents();
  const long long total = (long long)gridDim.x * 256;
  for (long long k = p.counts[0] + (long long)blockIdx.x * 256 + threadIdx.x;
       k < p.num_blocks / 2; k += total)
    p.src[k] = p.dst[k] = -1;
  const int row = blockIdx.x / per_row, y = blockIdx.x % per_row;
  if (row >= p.rows) return;
  const int n = p.ctx[row];
  if (n <= 0) return;
  const long long k = min((long long)ceil_div_blocks(n), p.stride);
  if (threadIdx.x == 0 && y == 0 && ceil_div_blocks(n) > p.stride) report(p.err, PA_DEVERR_SHAPE);
  for (long long j = y * 256 + threadIdx.x; j < k; j += per_row * 256) {
    const int page = p.tables[row * p.stride + j];
    if (page >= 0 && page < p.num_blocks)
      p.tables[row * p.stride + j] = p.remap[page];
    else
      report(p.err, PA_DEVERR_BLOCK_INDEX);
  }
}

// Blocks along a table row: enough that a block's 256 threads take few turns.
unsigned row_blocks(long long stride) {
  const long long y = (stride + 1023) / 1024;
  return (unsigned)(y < 1 ? 1 : y > 64 ? 64 : y);
}

// Whether any of the int32 arrays does not start on a 4-byte boundary.
template <typename... T>
bool misaligned4(const T *...x) {
  return ((reinterpret_cast<uintptr_t>(x) | ...) & 3) != 0;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_copy_pages(const pa_page_pool *pools, int32_t num_pools,
                                   int64_t num_blocks, const int32_t *src, const int32_t *dst,
                                   int32_t num_pairs, const int32_t *count, int32_t *error_flags,
                                   uint32_t flags, void *stream) {
  using namespace pa;
  if (num_pools < 0 || num_pairs < 0 || num_blocks < 0 || num_blocks > INT_MAX)
    return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (num_pools == 0 || num_pairs == 0) return PA_OK;
  if (!pools || !src || !dst) return PA_ERR_INVALID_ARG;
  if (misaligned4(src, dst, count, error_flags)) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i)
    if (!pools[i].base || pools[i].page_bytes < 1 || pools[i].page_bytes > (1ll << 31))
      return PA_ERR_INVALID_ARG;
  int device = -1, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return PA_ERR_DEVICE;
  for (int first = 0; first < num_pools; first += kCopyPools) {
    const int n = num_pools - first < kCopyPools ? num_pools - first : kCopyPools;
    CopyPagesParams p = {};
    p.num_blocks = num_blocks;
    p.src = src;
    p.dst = dst;
    p.num_pairs = num_pairs;
    p.count = count;
    p.err = error_flags;
    long long chunks = 0;
    for (int tiny = 0; tiny < 2; ++tiny)
      for (int i = 0; i < n; ++i) {
        const pa_page_pool &q = pools[first + i];
        if ((q.page_bytes <= 16) != (tiny == 1)) continue;
        const int at = p.num_big + p.num_tiny;
        p.pool[at].base = static_cast<uint8_t *>(q.base);
        p.pool[at].page_bytes = q.page_bytes;
        if (tiny) {
          ++p.num_tiny;
          continue;
        }
        chunks += (q.page_bytes + kCopyChunk - 1) / kCopyChunk;
        p.chunk_end[at] = (int)chunks;
        if ((reinterpret_cast<uintptr_t>(q.base) | (uintptr_t)q.page_bytes) % 16 == 0)
          p.vec[at >> 5] |= (int)(1u << (at & 31));
        ++p.num_big;
      }
    if (chunks > INT_MAX) return PA_ERR_UNSUPPORTED;
    const long long units = num_pairs * chunks + ((long long)num_pairs * p.num_tiny + 31) / 32;
    long long blocks = (units + kCopyWarps - 1) / kCopyWarps;
    if (blocks > 8ll * sms) blocks = 8ll * sms;
    if (launch_kernel(copy_pages_kernel, dim3((unsigned)blocks), dim3(32 * kCopyWarps), 0,
                      static_cast<cudaStream_t>(stream), true, p) != cudaSuccess)
      return PA_ERR_LAUNCH;
  }
  return PA_OK;
}

extern "C" pa_status pa_fork_pages(int32_t *block_tables, int32_t block_table_stride,
                                   int32_t *context_lens, int32_t num_rows,
                                   const int32_t *parents, const int32_t *children,
                                   int32_t num_forks, int32_t *ref_counts, int64_t num_blocks,
                                   int32_t block_size, int32_t *copy_src, int32_t *copy_dst,
                                   int32_t *forked, int32_t *error_flags, uint32_t flags,
                                   void *stream) {
  using namespace pa;
  if (num_rows < 0 || num_forks < 0 || num_blocks < 0 || num_blocks > INT_MAX)
    return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (num_forks == 0) return PA_OK;
  if (!block_tables || !context_lens || !parents || !children || !ref_counts || !copy_src ||
      !copy_dst || !forked || block_table_stride < 1)
    return PA_ERR_INVALID_ARG;
  if (misaligned4(block_tables, context_lens, parents, children, ref_counts, copy_src, copy_dst,
                  forked, error_flags))
    return PA_ERR_INVALID_ARG;
  ForkParams p{block_tables, block_table_stride, context_lens, num_rows, parents, children,
               num_forks, ref_counts, num_blocks, copy_src, copy_dst, forked, error_flags,
               (long long)num_forks * block_table_stride <= kInlineEntries};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_kernel(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s,
                    true, p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  if (!p.apply &&
      launch_kernel(fork_apply_kernel, dim3((unsigned)num_forks, row_blocks(block_table_stride)),
                    dim3(256), 0, s, true, p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}

extern "C" pa_status pa_free_pages(int32_t *block_tables, int32_t block_table_stride,
                                   int32_t *context_lens, int32_t num_rows, const int32_t *seqs,
                                   int32_t num_seqs, int32_t *ref_counts, int64_t num_blocks,
                                   int32_t block_size, int32_t *error_flags, uint32_t flags,
                                   void *stream) {
  using namespace pa;
  if (num_rows < 0 || num_seqs < 0 || num_blocks < 0 || num_blocks > INT_MAX)
    return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!block_tables || !context_lens || !seqs || !ref_counts || block_table_stride < 1)
    return PA_ERR_INVALID_ARG;
  if (misaligned4(block_tables, context_lens, seqs, ref_counts, error_flags))
    return PA_ERR_INVALID_ARG;
  if (launch_kernel(free_pages_kernel, dim3((unsigned)num_seqs), dim3(256), 0,
                    static_cast<cudaStream_t>(stream), true, block_tables,
                    (long long)block_table_stride, context_lens, (int)num_rows, seqs, ref_counts,
                    (long long)num_blocks, error_flags) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}

extern "C" pa_status pa_compact_pages(int32_t *block_tables, int32_t block_table_stride,
                                      const int32_t *context_lens, int32_t num_rows,
                                      int32_t *ref_counts, int64_t num_blocks, int32_t block_size,
                                      int32_t *copy_src, int32_t *copy_dst, int32_t *counts,
                                      int32_t *remap, int32_t *error_flags, uint32_t flags,
                                      void *stream) {
  using namespace pa;
  if (num_rows < 0 || num_blocks < 0 || num_blocks > INT_MAX) return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (!counts) return PA_ERR_INVALID_ARG;
  if (num_blocks > 0 && (!ref_counts || !remap)) return PA_ERR_INVALID_ARG;
  if (num_blocks > 1 && (!copy_src || !copy_dst)) return PA_ERR_INVALID_ARG;
  if (num_rows > 0 && (!block_tables || !context_lens || block_table_stride < 1))
    return PA_ERR_INVALID_ARG;
  if (misaligned4(block_tables, context_lens, ref_counts, copy_src, copy_dst, counts, remap,
                  error_flags))
    return PA_ERR_INVALID_ARG;
  CompactParams p{block_tables, block_table_stride, context_lens, num_rows, ref_counts,
                  num_blocks, copy_src, copy_dst, counts, remap, error_flags};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_kernel(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s,
                    true, p) != cudaSuccess)
    return PA_ERR_LAUNCH;
  const int per_row = (int)row_blocks(block_table_stride);
  const long long blocks = num_rows > 0 ? (long long)num_rows * per_row : 1;
  if (launch_kernel(compact_apply_kernel, dim3((unsigned)blocks), dim3(256), 0, s, true, p,
                    per_row) != cudaSuccess)
    return PA_ERR_LAUNCH;
  return PA_OK;
}
