// Rows of a paged cache close up: row first_i + r of sequence i's new block
// table becomes row positions_i[r] of its old one, K and V, for every KV head
// alike or with positions of its own per head.  After a step of speculative
// decoding the accepted drafts move to where the sequence goes on; after an
// eviction the rows that stay close up.
//
// Bound by bytes: each moved row is read and written once.  A CTA takes one
// sequence, KV head and operand (K or V) and chunks of rows of it; a thread
// keeps one 16-byte column of kRowsInFlight rows, the next chunk's rows on
// their way while the last one's are written.
//
// In place (new tables = old tables) a CTA walks all chunks of its rows in
// order.  That is safe wherever positions[r] >= first + r, in whatever order
// they are and however often: a chunk's rows are read before any of it is
// written (barrier), and rows written so far lie below first + (next chunk's
// first r), so no later chunk reads them.  Columns, heads and operands never
// meet.  Between different tables the chunks are independent and go to CTAs of
// their own.
//
// Measured: 16 rows of 4,096 to 16,384 tokens cut to 2,048 rows a KV head (8 of
// 128, bf16, fresh blocks), 269 MB read and written: see the table of cases.
#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kCompactThreads = 256;
constexpr int kRowsInFlight = 8;      // 16-byte loads of a thread in flight

// Byte offset of a sequence's row `pos` (one head) in either operand; -1 where
// the table has no such row.
__device__ __forceinline__ int64_t row_offset(const CompactArgs& a, const int32_t* __restrict__ table, int limit,
                                              int pos, int64_t head_off) {
  if (pos < 0 || pos >= limit) {
    flag_error(a.err, PKVD_ERR_CONTEXT);
    return -1;
  }
  const int b = __ldg(table + (pos >> a.block_shift));
  if (b < 0 || b >= a.num_blocks) {
    flag_error(a.err, PKVD_ERR_BLOCK_ID);
    return -1;
  }
  return ((int64_t)b * a.block_stride + (int64_t)(pos & (a.block_size - 1)) * a.token_stride + head_off) * a.elem_bytes;
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactArgs a) {
  pdl_wait();          // rows, positions and counts may come from the kernel before
  pdl_trigger();
  const int seq = blockIdx.y, head = blockIdx.x >> 1;
  uint8_t* base = static_cast<uint8_t*>(blockIdx.x & 1 ? a.v_base : a.k_base);
  const int per_row = a.head_dim * a.elem_bytes / 16;            // 8, 16 or 32 columns
  const int rows = kCompactThreads / per_row, r0 = threadIdx.x / per_row;
  const int64_t col = (threadIdx.x % per_row) * 16;
  const int64_t head_off = (int64_t)head * a.head_stride;
  const int32_t* pos = a.positions + (int64_t)seq * a.pos_stride + (int64_t)head * a.pos_head_stride;
  const int32_t* from = a.tables + (int64_t)seq * a.max_blocks;
  const int32_t* to = a.new_tables + (int64_t)seq * a.new_max_blocks;
  const int first = a.first ? a.first[seq] : 0;
  int n = a.counts[seq];
  if (n < 0 || n > a.max_count || first < 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) flag_error(a.err, PKVD_ERR_CONTEXT);
    if (first < 0) return;
    n = min(max(n, 0), a.max_count);
  }
  const int chunk = rows * kRowsInFlight;
  // the rows of the chunk from r on: where they lie, -1 for none
  auto sources = [&](int r, int64_t (&src)[kRowsInFlight]) {
    int p[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int at = r + i * rows + r0;
      p[i] = at < n ? pos[at] : -1;
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int at = r + i * rows + r0;
      src[i] = -1;
      if (at >= n) continue;
      if (IN_PLACE && p[i] < first + (int64_t)at) {              // would read a row already written
        flag_error(a.err, PKVD_ERR_CONTEXT);
        continue;
      }
      if (IN_PLACE && p[i] == first + (int64_t)at) continue;     // stays where it is
      src[i] = row_offset(a, from, a.max_tokens, p[i], head_off);
    }
  };
  int64_t src[kRowsInFlight];
  uint4 v[kRowsInFlight];
  const int step = IN_PLACE ? chunk : chunk * (int)gridDim.z;
  int r = IN_PLACE ? 0 : chunk * (int)blockIdx.z;
  if (r >= n) return;
  sources(r, src);
#pragma unroll
  for (int i = 0; i < kRowsInFlight; ++i)
    if (src[i] >= 0) v[i] = *reinterpret_cast<const uint4*>(base + src[i] + col);
  for (;;) {
    const int next = r + step;
    int64_t nsrc[kRowsInFlight];
    uint4 nv[kRowsInFlight];
    if (next < n) {
      sources(next, nsrc);
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i)
        if (nsrc[i] >= 0) nv[i] = *reinterpret_cast<const uint4*>(base + nsrc[i] + col);
    }
    if (IN_PLACE) __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      if (src[i] < 0) continue;
      const int64_t at = first + (int64_t)(r + i * rows + r0);
      const int64_t dst = row_offset(a, to, a.new_max_tokens, at > 0x7fffffff ? -1 : (int)at, head_off);
      if (dst >= 0) *reinterpret_cast<uint4*>(base + dst + col) = v[i];
    }
    if (next >= n) break;
    r = next;
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) src[i] = nsrc[i], v[i] = nv[i];
  }
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, int num_seqs, int num_kv_heads, cudaStream_t stream) {
  if (num_seqs == 0 || a.max_count == 0) return cudaSuccess;
  const int chunk = kCompactThreads * 16 / (a.head_dim * a.elem_bytes) * kRowsInFlight;
  if (a.new_tables == a.tables)
    return launch_pdl(compact_kernel<true>, dim3(num_kv_heads * 2, num_seqs), dim3(kCompactThreads), 0, stream, a);
  const int chunks = (a.max_count + chunk - 1) / chunk;
  return launch_pdl(compact_kernel<false>, dim3(num_kv_heads * 2, num_seqs, chunks < 65535 ? chunks : 65535),
                    dim3(kCompactThreads), 0, stream, a);
}

}  // namespace pkvd
