// Rows of a paged cache close up: row first_i + r of sequence i's new block
// table becomes row positions_i[r] of its old one, K and V, for every KV head
// alike or with positions of its own per head.  After a step of speculative
// decoding the accepted drafts move to where the sequence goes on; after an
// eviction the rows that stay close up.
//
// Bound by bytes: each moved row is read and written once.  A thread owns one
// 16-byte column (operand, head, part of the head) and takes kRowsInFlight rows
// of it at a time.
//
// In place (new tables = old tables) a CTA walks all rows of its columns in
// order.  That is safe wherever positions[r] >= first + r, in whatever order
// they are and however often: a chunk's rows are read before any of it is
// written, and rows written so far lie below first + (next chunk's first r), so
// no later chunk reads them.  Columns never meet.  Lists of up to kShort rows
// have one thread a column and need no barrier (256 sequences of up to 16 drafts,
// 8 heads of 128 in bf16: 7 us, 33 with the long lists' form); longer ones as many
// as fill the CTA, which meet at a barrier a chunk, the next chunk's rows on their
// way.  Between different tables the chunks are independent and go to CTAs of
// their own: 16 lists of up to 2,048 rows of their own for each of 8 heads, 270 MB
// to be moved, take 49 us, 0.82 of the copy rate (75 with two loads in flight).
#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsInFlight = 8;      // 16-byte loads of a thread in flight
constexpr int kShort = 32;

// Byte offset of a sequence's row `pos` in either operand, without the column; -1
// where the table has no such row.
__device__ __forceinline__ int64_t row_offset(const CompactArgs& a, const int32_t* __restrict__ table, int limit,
                                              int pos) {
  if (pos < 0 || pos >= limit) {
    flag_error(a.err, PKVD_ERR_CONTEXT);
    return -1;
  }
  const int b = __ldg(table + (pos >> a.block_shift));
  if (b < 0 || b >= a.num_blocks) {
    flag_error(a.err, PKVD_ERR_BLOCK_ID);
    return -1;
  }
  return ((int64_t)b * a.block_stride + (int64_t)(pos & (a.block_size - 1)) * a.token_stride) * a.elem_bytes;
}

enum : int { kFresh = 0, kInPlace = 1, kInPlaceShort = 2 };

template <int KIND>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  pdl_wait();          // rows, positions and counts may come from the kernel before
  pdl_trigger();
  const int seq = blockIdx.y;
  const int per_row = a.head_dim * a.elem_bytes / 16;            // 8, 16 or 32 columns of a head
  const int per_cta = KIND == kInPlaceShort ? kThreads : per_row;
  const int groups = kThreads / per_cta, r0 = threadIdx.x / per_cta;
  const int column = blockIdx.x * per_cta + threadIdx.x % per_cta;
  if (column >= 2 * a.num_kv_heads * per_row) return;            // (the short kind only: no barrier)
  const int part = column / per_row, head = part >> 1;
  uint8_t* base = static_cast<uint8_t*>(part & 1 ? a.v_base : a.k_base) +
                  (int64_t)head * a.head_stride * a.elem_bytes + (column % per_row) * 16;
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
  const int chunk = groups * kRowsInFlight;
  auto load = [&](int r, int64_t (&src)[kRowsInFlight], uint4 (&v)[kRowsInFlight]) {
    int p[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int at = r + i * groups + r0;
      p[i] = at < n ? pos[at] : -1;
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int at = r + i * groups + r0;
      src[i] = -1;
      if (at >= n) continue;
      if (KIND != kFresh && p[i] < first + (int64_t)at) {              // would read a row already written
        flag_error(a.err, PKVD_ERR_CONTEXT);
        continue;
      }
      if (KIND != kFresh && p[i] == first + (int64_t)at) continue;     // stays where it is
      src[i] = row_offset(a, from, a.max_tokens, p[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i)
      if (src[i] >= 0) v[i] = *reinterpret_cast<const uint4*>(base + src[i]);
  };
  auto store = [&](int r, const int64_t (&src)[kRowsInFlight], const uint4 (&v)[kRowsInFlight]) {
    int64_t dst[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
      const int64_t at = first + (int64_t)(r + i * groups + r0);
      dst[i] = src[i] < 0 ? -1 : row_offset(a, to, a.new_max_tokens, at > 0x7fffffff ? -1 : (int)at);
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i)
      if (dst[i] >= 0) *reinterpret_cast<uint4*>(base + dst[i]) = v[i];
  };
  int64_t src[kRowsInFlight];
  uint4 v[kRowsInFlight];
  if (KIND != kInPlace) {
    // a column's rows belong to one thread, or no row that is written is read
    const int step = KIND == kFresh ? chunk * (int)gridDim.z : chunk;
    for (int r = KIND == kFresh ? chunk * (int)blockIdx.z : 0; r < n; r += step) {
      load(r, src, v);
      store(r, src, v);
    }
    return;
  }
  if (n == 0) return;
  load(0, src, v);
  for (int r = 0;;) {
    const int next = r + chunk;
    int64_t nsrc[kRowsInFlight];
    uint4 nv[kRowsInFlight];
    if (next < n) load(next, nsrc, nv);
    __syncthreads();
    store(r, src, v);
    if (next >= n) break;
    r = next;
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) src[i] = nsrc[i], v[i] = nv[i];
  }
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0 || a.max_count == 0) return cudaSuccess;
  const int per_row = a.head_dim * a.elem_bytes / 16, columns = 2 * a.num_kv_heads * per_row;
  const int parts = 2 * a.num_kv_heads;
  if (a.new_tables == a.tables) {
    if (a.max_count <= kShort)
      return launch_pdl(compact_kernel<kInPlaceShort>, dim3((columns + kThreads - 1) / kThreads, num_seqs), dim3(kThreads), 0,
                        stream, a);
    return launch_pdl(compact_kernel<kInPlace>, dim3(parts, num_seqs), dim3(kThreads), 0, stream, a);
  }
  const int chunk = kThreads / per_row * kRowsInFlight, chunks = (a.max_count + chunk - 1) / chunk;
  return launch_pdl(compact_kernel<kFresh>, dim3(parts, num_seqs, chunks < 65535 ? chunks : 65535), dim3(kThreads), 0,
                    stream, a);
}

}  // namespace pkvd
