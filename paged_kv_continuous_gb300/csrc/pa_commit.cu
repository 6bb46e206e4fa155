// pa_commit_tree: the K/V rows of accepted nodes move up behind the committed keys,
// in every pool, and the sequences shrink to them.
//
// A cluster of CTAs takes a sequence.  A thread owns one 16-byte column of one
// pool's row and moves it for every step of the path in order, four loads ahead of
// their stores.  A path increases, so step i comes from node path[i] >= i: what
// a later step reads no earlier one has overwritten, in whatever order the columns
// run.  The slots of the path's steps (table lookups) are worked out once a CTA.
// context_lens changes behind a cluster barrier, when no CTA reads it any more.
//
// Bound by latency: a few hundred KB to move at most, behind five dependent loads.
#include <climits>

#include <cooperative_groups.h>

#include "pa_common.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

constexpr int kCmThreads = 256;
constexpr int kCmRanks = 8;    // CTAs of a cluster
constexpr int kCmPools = 128;  // pools per launch
constexpr int kCmSteps = 256;  // steps of a path at a time

struct CommitPool {
  uint8_t *base;
  long long row_bytes;
};
struct CommitParams {
  CommitPool pool[kCmPools];
  int column_end[kCmPools];  // columns of pools 0 .. i
  int wide[kCmPools / 32];   // bit i: columns of 16 bytes, else of one
  int num_pools;
  long long num_blocks;
  const int32_t *tables;
  long long bt_stride;
  int32_t *ctx;
  const int32_t *cu;
  const int32_t *path;
  long long path_stride;
  const int32_t *accepted;
  int32_t *refs;
  int last;  // this launch ends the call: lengths and counts follow
  int32_t *err;
};

template <typename T>
__device__ __forceinline__ void move_column(uint8_t *base, long long row_bytes, const int *src,
                                            const int *dst, int n) {
  constexpr int kAhead = 4;
  for (int i = 0; i < n; i += kAhead) {
    T v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k < n && src[i + k] >= 0)
        v[k] = *reinterpret_cast<const T *>(base + src[i + k] * row_bytes);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k < n && src[i + k] >= 0) *reinterpret_cast<T *>(base + dst[i + k] * row_bytes) = v[k];
  }
}

__global__ void __launch_bounds__(kCmThreads)
    commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int from[kCmSteps], to[kCmSteps];  // slots; from -1: nothing to move
  cg::cluster_group cluster = cg::this_cluster();
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int rank = (int)cluster.block_rank(), seq = (int)blockIdx.x / kCmRanks;
  const bool tell = rank == 0 && p.last;
  const int keys = p.ctx[seq], count = p.accepted[seq];
  const long long nodes = (long long)p.cu[seq + 1] - p.cu[seq];
  const int32_t *path = p.path + seq * p.path_stride;
  const int32_t *row = p.tables + seq * p.bt_stride;
  bool bad = nodes < 0 || (nodes > 0 && (nodes > keys || ceil_div_blocks(keys) > p.bt_stride)) ||
             count < 0 || count > nodes || count > p.path_stride;
  if (!bad)
    for (int i = tid; i < count; i += kCmThreads) {
      const int a = path[i];
      bad |= a < 0 || a >= nodes || (i > 0 && a <= path[i - 1]);
    }
  bad = __syncthreads_or(bad);
  if (bad || nodes == 0) {  // (the whole cluster)
    if (bad && tell && tid == 0) report(p.err, PA_DEVERR_SHAPE);
    return;
  }
  const int done = keys - (int)nodes;
  const int columns = p.num_pools ? p.column_end[p.num_pools - 1] : 0;
  for (int i0 = 0; i0 < count; i0 += kCmSteps) {
    const int n = min(kCmSteps, count - i0);
    if (i0) __syncthreads();
    for (int i = tid; i < n; i += kCmThreads) {
      const int a = done + path[i0 + i], b = done + i0 + i;
      int src = -1, dst = -1;
      if (a != b) {
        const int pa = row[a / kBlockSize], pb = row[b / kBlockSize];
        if (pa < 0 || pa >= p.num_blocks || pb < 0 || pb >= p.num_blocks) {
          if (tell) report(p.err, PA_DEVERR_BLOCK_INDEX);
        } else {
          src = pa * kBlockSize + a % kBlockSize;
          dst = pb * kBlockSize + b % kBlockSize;
        }
      }
      from[i] = src;
      to[i] = dst;
    }
    __syncthreads();
    for (int c = rank * kCmThreads + tid; c < columns; c += kCmRanks * kCmThreads) {
      int lo = 0, hi = p.num_pools - 1;  // the pool: the first whose columns end past c
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (c < p.column_end[mid])
          hi = mid;
        else
          lo = mid + 1;
      }
      const long long col = c - (lo ? p.column_end[lo - 1] : 0);
      const CommitPool q = p.pool[lo];
      if ((p.wide[lo >> 5] >> (lo & 31)) & 1)
        move_column<uint4>(q.base + 16 * col, q.row_bytes, from, to, n);
      else
        move_column<uint8_t>(q.base + col, q.row_bytes, from, to, n);
    }
  }
  if (!p.last) return;
  cluster.sync();  // every CTA has read the old length
  if (rank != 0) return;
  if (tid == 0) p.ctx[seq] = done + count;
  if (!p.refs) return;
  const int e0 = ceil_div_blocks(done + count), e1 = ceil_div_blocks(keys);
  for (int e = e0 + tid; e < e1; e += kCmThreads) {
    const int page = row[e];
    if (page < 0 || page >= p.num_blocks) {
      report(p.err, PA_DEVERR_BLOCK_INDEX);
    } else if (atomicSub(p.refs + page, 1) < 1) {
      atomicAdd(p.refs + page, 1);
      report(p.err, PA_DEVERR_PAGES);
    }
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_commit_tree(const pa_page_pool *pools, int32_t num_pools,
                                    int64_t num_blocks, const int32_t *block_tables,
                                    int32_t block_table_stride, int32_t *context_lens,
                                    const int32_t *cu_seqlens, int32_t num_seqs,
                                    const int32_t *path, int32_t path_stride,
                                    const int32_t *accepted, int32_t *ref_counts,
                                    int32_t block_size, int32_t *error_flags, uint32_t flags,
                                    void *stream) {
  using namespace pa;
  if (num_pools < 0 || num_seqs < 0 || num_blocks < 0 || path_stride < 0) return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (num_blocks < 1 || num_blocks > INT_MAX / kBlockSize || block_table_stride < 1)
    return PA_ERR_INVALID_ARG;
  if (num_seqs > INT_MAX / kCmRanks) return PA_ERR_UNSUPPORTED;
  if (!block_tables || !context_lens || !cu_seqlens || !accepted || (num_pools > 0 && !pools) ||
      (path_stride > 0 && !path))
    return PA_ERR_INVALID_ARG;
  for (const void *x : {(const void *)block_tables, (const void *)context_lens,
                        (const void *)cu_seqlens, (const void *)path, (const void *)accepted,
                        (const void *)ref_counts, (const void *)error_flags})
    if (reinterpret_cast<uintptr_t>(x) & 3) return PA_ERR_INVALID_ARG;
  for (int i = 0; i < num_pools; ++i)
    if (!pools[i].base || pools[i].page_bytes < 1 || pools[i].page_bytes > (1ll << 31) ||
        pools[i].page_bytes % kBlockSize)
      return PA_ERR_INVALID_ARG;
  CommitParams p = {};
  p.num_blocks = num_blocks;
  p.tables = block_tables;
  p.bt_stride = block_table_stride;
  p.ctx = context_lens;
  p.cu = cu_seqlens;
  p.path = path;
  p.path_stride = path_stride;
  p.accepted = accepted;
  p.refs = ref_counts;
  p.err = error_flags;
  int next = 0;
  do {
    long long columns = 0;
    p.num_pools = 0;
    for (int &w : p.wide) w = 0;
    while (next < num_pools && p.num_pools < kCmPools) {
      const long long bytes = pools[next].page_bytes / kBlockSize;
      const bool wide = (reinterpret_cast<uintptr_t>(pools[next].base) | (uintptr_t)bytes) % 16 == 0;
      const long long more = wide ? bytes / 16 : bytes;
      if (columns + more > INT_MAX - kCmRanks * kCmThreads) break;  // (never the first pool)
      const int i = p.num_pools++;
      columns += more;
      p.pool[i] = {static_cast<uint8_t *>(pools[next].base), bytes};
      p.column_end[i] = (int)columns;
      if (wide) p.wide[i >> 5] |= (int)(1u << (i & 31));
      ++next;
    }
    p.last = next == num_pools;
    if (launch_cluster(commit_kernel, dim3((unsigned)num_seqs * kCmRanks), dim3(kCmThreads),
                       kCmRanks, 0, static_cast<cudaStream_t>(stream), p) != cudaSuccess)
      return PA_ERR_LAUNCH;
  } while (next < num_pools);
  return PA_OK;
}
