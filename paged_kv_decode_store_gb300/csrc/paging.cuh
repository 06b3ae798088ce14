// Where a new token goes: its position in its sequence and its slot in the
// paged cache, for decode rows (context lengths) and for the rows of a varlen
// prefill batch (cu_seqlens_q / cu_seqlens_k).  Shared by the store kernels
// (store.cu) and the rotary store kernels (rope.cu).
#pragma once

#include "common.cuh"

namespace pkvd {

// position -1: the row has none (inactive, past the batch, or a bad length,
// which is flagged).  slot -1: nothing is stored (also for a position past
// the table or a bad block id, which are flagged).
struct TokenPlace {
  int pos;
  int64_t slot;
};

// Slot of position `pos` through one row of the block table.
__device__ __forceinline__ int64_t slot_of(const int32_t* __restrict__ table, int max_blocks, int pos,
                                           int block_size, int64_t num_blocks, int32_t* err) {
  const int logical = pos / block_size;
  if (logical >= max_blocks) {
    flag_error(err, PKVD_ERR_CONTEXT);
    return -1;
  }
  const int phys = table[logical];
  if (phys < 0 || phys >= num_blocks) {
    flag_error(err, PKVD_ERR_BLOCK_ID);
    return -1;
  }
  return (int64_t)phys * block_size + pos % block_size;
}

// Row i's newest token: position context_len - 1.
__device__ __forceinline__ TokenPlace decode_place(const int32_t* __restrict__ tables, int max_blocks,
                                                   const int32_t* __restrict__ ctx, int i, int block_size,
                                                   int64_t num_blocks, int32_t* err) {
  const int c = ctx[i];
  if (c <= 0) {
    if (c < 0) flag_error(err, PKVD_ERR_CONTEXT);
    return {-1, -1};
  }
  return {c - 1, slot_of(tables + (int64_t)i * max_blocks, max_blocks, c - 1, block_size, num_blocks, err)};
}

// New token row t of a varlen prefill batch.  nano-vllm "Model Runner" notes,
// section "prefix cache": sequence i owns rows [cu_q[i], cu_q[i+1]) and k_len
// = cu_k[i+1] - cu_k[i] tokens in all, so row t sits at position (k_len -
// q_len) + (t - cu_q[i]).
__device__ __forceinline__ TokenPlace prefill_place(const int32_t* __restrict__ tables, int max_blocks,
                                                    const int32_t* __restrict__ cu_q, const int32_t* __restrict__ cu_k,
                                                    int num_seqs, int t, int block_size, int64_t num_blocks,
                                                    int32_t* err) {
  if (t >= cu_q[num_seqs]) return {-1, -1};
  int lo = 0, hi = num_seqs - 1;   // the last i with cu_q[i] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu_q[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int q0 = cu_q[lo], q1 = cu_q[lo + 1];
  const int qlen = q1 - q0, klen = cu_k[lo + 1] - cu_k[lo];
  if (t < q0 || t >= q1 || klen < qlen) {
    flag_error(err, PKVD_ERR_CONTEXT);
    return {-1, -1};
  }
  const int pos = klen - qlen + (t - q0);
  return {pos, slot_of(tables + (int64_t)lo * max_blocks, max_blocks, pos, block_size, num_blocks, err)};
}

}  // namespace pkvd
