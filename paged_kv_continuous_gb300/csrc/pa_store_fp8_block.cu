// pa_store_kv_fp8_block: appends the new K/V rows of packed sequences to a
// block-scaled FP8 cache (pa_fp8_block.cuh).  The chunk of sequence s covers
// positions context_lens[s] - q_len .. context_lens[s] - 1; for each page it
// touches, each kv head, and K and V apart, with r0 .. r1 - 1 the page's rows
// it writes and a the largest finite |x| of them:
//   e     = smallest e with a <= 448 * 2^e, not below the page's scale so far
//           when rows before r0 stay (r0 > 0);
//   code  = E4M3(x * 2^-e), nearest even, for the new rows;
//   code' = E4M3(code * 2^(e_old - e)) for the rows before r0, if e grew.
//
// One warp takes one (page, kv head) of K or of V: 16 rows x 128 dims.  Lane
// L owns dims 4L .. 4L + 3 of every row, so a row load is 256 contiguous
// bytes of the warp, all the page's loads are in flight together, and the
// maximum is one warp reduction.  K codes leave as 128-byte token rows; V
// pages are dim-major ([128 dims][16 tokens]), where a lane's four dims are
// four 16-byte rows: 2 KB per warp, contiguous.  The scale is a power of two,
// so x * 2^-e is exact in fp32 and each code is rounded once.
//
// Work list.  A sequence of q tokens touches at most floor(q / 16) + 2 pages,
// so unit u = floor(cu_seqlens[s] / 16) + 2 s + i names the i-th page of
// sequence s without overlap, the host sizes the grid from total_tokens and
// num_seqs alone, and a warp finds its s by a 32-way search.  A chunk that is not
// consistent may have no unit, so warps behind the units look at all sequences,
// one per lane, and report.
//
// Measured in chains of calls: 5 x 5-8 k tokens at 8 kv heads (204 MB) 33.9 us,
// 6.0 TB/s, 89 % of the measured copy bandwidth; 32 k tokens at 2 kv heads (49 MB)
// 9.5 us; the 64 tokens of a decode step 3.6 us (launch and four dependent
// loads).  It was
// bound by its instructions, not by memory: pages that are all new take a path
// without row masks, two bf16 per maximum and byte transposes of two rounds of
// permutes (about 280 instructions a warp, from 700), 45.3 -> 34.1 us.  A warp
// that fetches its next page's rows while it codes one (half the warps fit) was
// slower, 51.6 us.
#include "pa_fp8_block.cuh"

namespace pa {
namespace {

constexpr int kQsWarps = 4;

struct QuantStoreParams {
  const uint16_t *rows[2];  // K, V
  long long tok[2], head[2];
  uint8_t *cache[2];
  uint8_t *scale[2];
  long long num_blocks;
  int hkv;
  const int32_t *cu_seqlens;
  int num_seqs;
  int total_tokens;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int32_t *err;
  long long units;
};

// First unit of sequence s.
__device__ __forceinline__ long long first_unit(const int32_t *cu, int s) {
  return (long long)(cu[s] >> 4) + 2ll * s;
}

// The sequence whose units hold u: the largest s with first_unit(s) <= u, by
// a 32-way search over all lanes (two rounds of loads up to 1024 sequences).
__device__ __forceinline__ int find_seq(const int32_t *cu, int num_seqs, long long u, int lane) {
  int lo = 0, n = num_seqs;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int s = lo + min(lane * step, n - 1);
    const unsigned m = __ballot_sync(0xffffffffu, first_unit(cu, s) <= u);
    // cu_seqlens may be inconsistent: any answer is in range
    const int top = m ? 31 - __clz(m) : 0;
    const int from = min(top * step, n - 1);
    lo += from;
    n = min(step, n - from);
  }
  return lo;
}

// A chunk cu_seqlens[s] = c0 .. c1 - 1 that lies outside the rows or is longer than
// its context n.
__device__ __forceinline__ bool inconsistent(int c0, int c1, int n, int total_tokens) {
  return c0 < 0 || c1 < c0 || c1 > total_tokens || n < c1 - c0;
}

// One warp's share of a page: rows r0 .. r1 - 1 of one head of K (dst = row 0 of
// the head) or V (dst = the lane's first dim row).
struct Share {
  const uint16_t *src;  // row 0 of the page in k / v, the lane's dims
  long long tok;        // stride of a token in elements
  uint8_t *dst, *scale;
  long long k_row;      // bytes from one K row of the head to the next
  int r0, r1;
};

// kFull: all 16 rows are new, and nothing the page holds matters.
template <bool kFull, bool kIsV>
__device__ __forceinline__ void store_share(const Share &t, const uint2 (&row)[kBlockSize]) {
  const int r0 = kFull ? 0 : t.r0, r1 = kFull ? kBlockSize : t.r1;
  const int old =
      !kFull && r0 > 0 ? min(max((int)*t.scale, kScaleMin), kScaleMax) : 0;
  uint4 vold[4];
  if (kIsV && !kFull) {
#pragma unroll
    for (int d = 0; d < 4; ++d) vold[d] = *reinterpret_cast<const uint4 *>(t.dst + d * kBlockSize);
  }

  // ---- the page's scale ------------------------------------------------------
  // |x| of bf16 orders like its bits (two elements per maximum).  Infinities
  // and NaN (exponent all ones) do not count -- an infinity saturates, a NaN
  // keeps its code -- so where the warp met one it looks again, without them.
  uint32_t top2 = 0;
#pragma unroll
  for (int r = 0; r < kBlockSize; ++r)
    top2 = __vmaxu2(top2, __vmaxu2(row[r].x & 0x7FFF7FFFu, row[r].y & 0x7FFF7FFFu));
  uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 >> 16, top2 & 0xFFFFu));
  if (top >= 0x7F80u) {
    top = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      const uint16_t *q = t.src + (long long)r * t.tok;
      for (int k = 0; k < 4; ++k) {
        const uint32_t a = q[k] & 0x7FFFu;
        top = max(top, a < 0x7F80u ? a : 0u);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const int e = max(scale_for(__uint_as_float(top << 16)), old);
  const float inv = inv_scale_of(e);
  const bool grew = !kFull && r0 > 0 && e > old;
  const float down = grew ? __uint_as_float((uint32_t)(old - e + kScaleBias) << 23) : 1.f;

  // ---- the codes ---------------------------------------------------------------
  uint32_t code[kBlockSize];
#pragma unroll
  for (int r = 0; r < kBlockSize; ++r) {
    const float2 a = bf16x2_to_float2(row[r].x), b = bf16x2_to_float2(row[r].y);
    code[r] = e4m3x2_of(a.x * inv, a.y * inv) | (e4m3x2_of(b.x * inv, b.y * inv) << 16);
  }
  if (!kIsV) {
#pragma unroll
    for (int r = 0; r < kBlockSize; ++r) {
      uint32_t *q = reinterpret_cast<uint32_t *>(t.dst + r * t.k_row);
      if (kFull || (r >= r0 && r < r1))
        *q = code[r];
      else if (grew && r < r0)
        *q = recode4(*q, down);
    }
  } else {
    // rows to columns: the 16-byte dim row d holds byte d of every token's
    // codes; 4 x 4 bytes at a time, two rounds of byte permutes
    uint32_t o[4][4];  // [dim][tokens 4 q .. 4 q + 3]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a = code[4 * q], b = code[4 * q + 1], c = code[4 * q + 2], d = code[4 * q + 3];
      const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
      const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
      o[0][q] = __byte_perm(ab0, cd0, 0x5410);
      o[1][q] = __byte_perm(ab0, cd0, 0x7632);
      o[2][q] = __byte_perm(ab1, cd1, 0x5410);
      o[3][q] = __byte_perm(ab1, cd1, 0x7632);
    }
    if (!kFull) {
      // tokens past the chunk keep their bytes, earlier ones their values
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // bytes [r0, r1) of the page that fall in this word
        const int b0 = min(max(r0 - 4 * q, 0), 4), b1 = min(max(r1 - 4 * q, 0), 4);
        const uint32_t below = b0 >= 4 ? 0xFFFFFFFFu : (1u << (8 * b0)) - 1u;
        const uint32_t upto = b1 >= 4 ? 0xFFFFFFFFu : (1u << (8 * b1)) - 1u;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t kept = q == 0 ? vold[d].x : q == 1 ? vold[d].y : q == 2 ? vold[d].z : vold[d].w;
          if (grew) kept = (recode4(kept, down) & below) | (kept & ~below);
          o[d][q] = (o[d][q] & upto & ~below) | (kept & ~(upto & ~below));
        }
      }
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
      *reinterpret_cast<uint4 *>(t.dst + d * kBlockSize) =
          make_uint4(o[d][0], o[d][1], o[d][2], o[d][3]);
  }
  if ((threadIdx.x & 31) == 0) *t.scale = (uint8_t)e;
}

template <bool kVec>
__global__ void __launch_bounds__(32 * kQsWarps, 8)
    store_kv_fp8_block_kernel(const QuantStoreParams p) {
  // Always a programmatic dependent: it waits for the kernel before first of
  // all, so only its set-up moves ahead.  Plain loads, not the read-only path:
  // that kernel may have written any of it while this one was set up.
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long w =
      (long long)blockIdx.x * kQsWarps + __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int per = 2 * p.hkv;
  const long long u = w / per;
  const int x = (int)(w % per), is_v = x & 1, h = x >> 1;
  if (u >= p.units) {
    const long long m = 32 * (u - p.units) + lane;
    if (x == 0 && m < p.num_seqs &&
        inconsistent(p.cu_seqlens[m], p.cu_seqlens[m + 1], p.context_lens[m], p.total_tokens))
      report(p.err, PA_DEVERR_SHAPE);
    return;
  }

  int s, c0, c1, n;
  if (p.num_seqs <= 32) {
    // one round of loads: a sequence per lane
    const int mine = min(lane, p.num_seqs - 1);
    const int a = p.cu_seqlens[mine], b = p.cu_seqlens[mine + 1];
    const int c = p.context_lens[mine];
    const unsigned m = __ballot_sync(0xffffffffu, (long long)(a >> 4) + 2ll * mine <= u);
    s = m ? min(31 - __clz(m), p.num_seqs - 1) : 0;
    c0 = __shfl_sync(0xffffffffu, a, s);
    c1 = __shfl_sync(0xffffffffu, b, s);
    n = __shfl_sync(0xffffffffu, c, s);
  } else {
    s = find_seq(p.cu_seqlens, p.num_seqs, u, lane);
    c0 = p.cu_seqlens[s];
    c1 = p.cu_seqlens[s + 1];
    n = p.context_lens[s];
  }
  const long long i = u - (((long long)(c0 >> 4)) + 2ll * s);  // page of the chunk
  if (inconsistent(c0, c1, n, p.total_tokens)) return;
  const int first = n - (c1 - c0);         // position of the chunk's first token
  const long long j = (first >> 4) + i;    // logical page
  if (c1 == c0 || i < 0 || j * kBlockSize >= n) return;
  if (j >= p.bt_stride) {
    if (x == 0 && lane == 0) report(p.err, PA_DEVERR_SHAPE);
    return;
  }
  // (requested before the rows and looked at after: one round of loads)
  const long long page = p.block_tables[(long long)s * p.bt_stride + j];
  const int base = (int)(j * kBlockSize);
  Share t;
  t.tok = p.tok[is_v];
  t.r0 = max(0, first - base);
  t.r1 = min(kBlockSize, n - base);
  t.src = p.rows[is_v] + (long long)(c0 + base - first) * t.tok + (long long)h * p.head[is_v] +
          4 * lane;
  uint2 row[kBlockSize];
#pragma unroll
  for (int r = 0; r < kBlockSize; ++r) {
    row[r] = make_uint2(0u, 0u);
    if (r >= t.r0 && r < t.r1) {
      const uint16_t *q = t.src + (long long)r * t.tok;
      if (kVec) {
        row[r] = __ldcs(reinterpret_cast<const uint2 *>(q));  // read once
      } else {
        row[r].x = (uint32_t)q[0] | ((uint32_t)q[1] << 16);
        row[r].y = (uint32_t)q[2] | ((uint32_t)q[3] << 16);
      }
    }
  }
  if (page < 0 || page >= p.num_blocks) {
    if (x == 0 && lane == 0) report(p.err, PA_DEVERR_BLOCK_INDEX);
    return;
  }
  t.scale = p.scale[is_v] + page * p.hkv + h;
  t.k_row = (long long)p.hkv * kHeadDim;
  t.dst = is_v ? p.cache[1] + ((page * p.hkv + h) * kHeadDim + 4 * lane) * kBlockSize
               : p.cache[0] + (page * kBlockSize * p.hkv + h) * kHeadDim + 4 * lane;
  const bool full = t.r0 == 0 && t.r1 == kBlockSize;
  if (is_v) {
    if (full)
      store_share<true, true>(t, row);
    else
      store_share<false, true>(t, row);
  } else {
    if (full)
      store_share<true, false>(t, row);
    else
      store_share<false, false>(t, row);
  }
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_store_kv_fp8_block(
    const void *k, const void *v, int64_t k_tok_stride, int64_t k_head_stride,
    int64_t v_tok_stride, int64_t v_head_stride, const int32_t *cu_seqlens, int32_t num_seqs,
    int32_t total_tokens, void *k_cache, void *v_cache, uint8_t *k_scale, uint8_t *v_scale,
    int64_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
    const int32_t *block_tables, int32_t block_table_stride, const int32_t *context_lens,
    int32_t *error_flags, uint32_t flags, void *stream) {
  using namespace pa;
  if (num_seqs < 0 || total_tokens < 0 || num_blocks < 0) return PA_ERR_INVALID_ARG;
  if (flags & ~static_cast<uint32_t>(PA_LAUNCH_PDL)) return PA_ERR_INVALID_ARG;
  if (head_dim != kHeadDim || block_size != kBlockSize) return PA_ERR_UNSUPPORTED;
  if (num_kv_heads < 1 || num_kv_heads > 64) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_tokens == 0) return PA_OK;
  if (!k || !v || !cu_seqlens || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables ||
      !context_lens)
    return PA_ERR_INVALID_ARG;
  if (block_table_stride < 1) return PA_ERR_INVALID_ARG;
  if (k_tok_stride < 0 || k_head_stride < 0 || v_tok_stride < 0 || v_head_stride < 0)
    return PA_ERR_INVALID_ARG;
  auto addr = [](const void *x) { return reinterpret_cast<uintptr_t>(x); };
  if ((addr(k_cache) | addr(v_cache)) % 16 || (addr(k) | addr(v)) % 2) return PA_ERR_INVALID_ARG;
  QuantStoreParams p;
  p.rows[0] = static_cast<const uint16_t *>(k);
  p.rows[1] = static_cast<const uint16_t *>(v);
  p.tok[0] = k_tok_stride;
  p.tok[1] = v_tok_stride;
  p.head[0] = k_head_stride;
  p.head[1] = v_head_stride;
  p.cache[0] = static_cast<uint8_t *>(k_cache);
  p.cache[1] = static_cast<uint8_t *>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.num_blocks = num_blocks;
  p.hkv = num_kv_heads;
  p.cu_seqlens = cu_seqlens;
  p.num_seqs = num_seqs;
  p.total_tokens = total_tokens;
  p.block_tables = block_tables;
  p.bt_stride = block_table_stride;
  p.context_lens = context_lens;
  p.err = error_flags;
  p.units = (long long)(total_tokens / kBlockSize) + 2ll * num_seqs;
  const long long warps = (p.units + (num_seqs + 31ll) / 32) * 2 * num_kv_heads;
  const long long blocks = (warps + kQsWarps - 1) / kQsWarps;
  if (blocks > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  // rows are read 8 bytes a lane where base and strides allow it
  const bool vec = ((addr(k) | addr(v)) % 8 == 0) && k_tok_stride % 4 == 0 &&
                   k_head_stride % 4 == 0 && v_tok_stride % 4 == 0 && v_head_stride % 4 == 0;
  const cudaError_t e = launch_kernel(
      vec ? store_kv_fp8_block_kernel<true> : store_kv_fp8_block_kernel<false>,
      dim3((unsigned)blocks), dim3(32 * kQsWarps), 0, static_cast<cudaStream_t>(stream),
      true, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_LAUNCH;
}
