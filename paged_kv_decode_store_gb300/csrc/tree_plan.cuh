// Attention of drafted trees: how its work is cut, shared by the kernels that
// compute it (tree.cu in fp32, tree_tc.cu on the tensor cores) and the merge.
//
// Sequence i has n_i drafted rows behind cached_i = k_len_i - n_i cached tokens.
// A unit is a run of its nodes (all query heads of one KV head: unit_rows
// rows); a unit, KV head and tile of 128 keys is the smallest piece of work.
// The pieces of the batch, sequence by sequence, unit by unit, head by head,
// tile by tile, are one list; slices of equal length go to the CTAs.  A CTA
// whose slice holds a (unit, head)'s tiles in part leaves a record (sums,
// maximum, sum of weights), which the merge kernel joins; whole ones are
// written at once.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkvd {

constexpr int kOwnSeqs = 128;               // batches of at most as many: every CTA finds its own slice

struct TreePlan {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int num_seqs, total_q, max_q, words;      // words: 32 ancestors each
  int unit_tokens, unit_rows;
  int hkv, hq, group;
  int window;
  int64_t table_tokens;                     // tokens a block table can hold
  int grid;                                 // CTAs; slices are at most as many
  // the workspace
  int64_t* starts;                          // [num_seqs + 1]: pieces before a sequence
  struct TreeStart* slice;                  // [grid]: where a slice begins
  struct TreeJoin* join;                    // [grid]: what is to be joined across a slice's begin
  int planned;                              // the plan kernel ran: starts and slice are there, and (for tree_tc.cu)
  uint32_t* anc;                            // [num_seqs][max_q][words]: a node's visible ancestors and itself, a bit each
  int32_t* depth;                           // [num_seqs][max_q]
  float* rec;                               // [2 grid][unit_rows][D]: sums of a slice's first and last segment
  float2* rec_ml;                           // [2 grid][unit_rows]: maximum (log2 units), sum of weights
};

struct TreeSeq {
  int q0, n, klen, cached;
  int lo, lo_tile, tiles, units;            // first key any node sees, its tile, tiles of keys, units
  __device__ int64_t pieces(int hkv) const { return (int64_t)units * hkv * tiles; }
};

__device__ __forceinline__ TreeSeq tree_seq(const TreePlan& p, int q0, int n, int klen) {
  TreeSeq s;
  s.q0 = q0;
  s.n = n;
  s.klen = klen;
  s.cached = s.klen - s.n;
  s.units = s.tiles = s.lo = s.lo_tile = 0;
  // (not by the sign of cached: a length near -2^31 minus n is a large number again)
  const bool ok = s.q0 >= 0 && s.n >= 0 && s.n <= p.max_q && s.klen >= s.n && (int64_t)s.q0 + s.n <= p.total_q &&
                  s.klen <= p.table_tokens;
  if (!ok) s.n = -1;
  if (s.n <= 0) return s;
  s.lo = p.window > 0 ? max(0, s.cached + 1 - p.window) : 0;
  s.lo_tile = s.lo / kTreeKeys;
  s.tiles = (s.klen - 1) / kTreeKeys - s.lo_tile + 1;
  s.units = s.n <= p.unit_tokens ? 1 : (s.n + p.unit_tokens - 1) / p.unit_tokens;
  return s;
}

__device__ __forceinline__ TreeSeq tree_seq(const TreePlan& p, int i) {
  return tree_seq(p, p.cu_q[i], p.cu_q[i + 1] - p.cu_q[i], p.cu_k[i + 1] - p.cu_k[i]);
}

// Slices of a batch of `total` pieces, and where one begins.
__device__ __forceinline__ int64_t tree_slices(const TreePlan& p, int64_t total) {
  return total < p.grid ? total : p.grid;
}
// (in 32 bits where they hold it -- slices are fewer than 2^10 -- because a 64-bit
// division takes hundreds of clocks)
__device__ __forceinline__ int64_t tree_slice_begin(int64_t total, int64_t slices, int64_t c) {
  return total < (1 << 22) ? (uint32_t)total * (uint32_t)c / (uint32_t)slices : total * c / slices;
}
// The slice that holds piece f.
__device__ __forceinline__ int64_t tree_slice_of(int64_t total, int64_t slices, int64_t f) {
  return total < (1 << 22) ? ((uint32_t)(f + 1) * (uint32_t)slices - 1u) / (uint32_t)total : ((f + 1) * slices - 1) / total;
}

// Where a slice begins, as the plan kernel leaves it: one load instead of a
// search and the sequence's lengths.
struct __align__(16) TreeStart {
  int64_t at, end;                          // the slice's pieces
  int64_t in;                               // the first one's place in its sequence
  int seq, q0;
  int n, klen;
  int pad[2];
};

// The same found by a warp, without the plan: from the lengths alone, which are
// inputs, so before the wait for the kernel before.  One launch less, 3 us of a
// small call; and short code, because a kernel's first instructions come from far.
struct OwnStart {
  int64_t total;                            // pieces in all
  TreeStart first;
  bool bad;                                 // one of them has lengths that cannot be
  __device__ OwnStart(const TreePlan& p, int c, int lane) {
    int64_t before[4], mine[4];             // pieces before sequences lane, lane + 32, .., and of them
    total = 0;
    bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      before[e] = mine[e] = 0;
      if (e * 32 >= p.num_seqs) continue;
      const int i = e * 32 + lane;
      if (i < p.num_seqs) {
        const TreeSeq s = tree_seq(p, i);
        bad |= s.n < 0;
        mine[e] = s.pieces(p.hkv);
      }
      int64_t upto = mine[e];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(FULL_MASK, upto, o);
        if (lane >= o) upto += t;
      }
      before[e] = total + upto - mine[e];
      total += __shfl_sync(FULL_MASK, upto, 31);
    }
    const int64_t slices = tree_slices(p, total);
    first.at = first.end = first.in = 0;
    first.seq = first.q0 = first.n = first.klen = 0;
    if (c >= slices) return;                // no piece for this CTA
    first.at = tree_slice_begin(total, slices, c);
    first.end = tree_slice_begin(total, slices, c + 1);
    int at = -1;                            // the sequence that has the first piece
    int64_t in = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (before[e] <= first.at && first.at < before[e] + mine[e]) at = e * 32 + lane, in = first.at - before[e];
    const int src = __ffs(__ballot_sync(FULL_MASK, at >= 0)) - 1;
    first.in = __shfl_sync(FULL_MASK, in, src);
    first.seq = __shfl_sync(FULL_MASK, at, src);
    first.q0 = p.cu_q[first.seq];
    first.n = p.cu_q[first.seq + 1] - first.q0;
    first.klen = p.cu_k[first.seq + 1] - p.cu_k[first.seq];
  }
};

// One segment of a slice: tiles [t0, t1) of a (unit, head).
struct TreeSegment {
  int seq, unit, head;
  int t0, t1;
  int slot;                                 // of its record; -1: the whole (unit, head)
};

// Walks a slice's segments.
struct TreeWalk {
  int64_t at, end, begin, in;               // in: `at` within its sequence
  int cta, seq;
  TreeSeq s;
  __device__ void start(const TreePlan& p, int c, const TreeStart& f) {
    cta = c;
    at = begin = f.at;
    end = f.end;
    in = f.in;
    seq = f.seq;
    s = tree_seq(p, f.q0, f.n, f.klen);
  }
  __device__ bool next(const TreePlan& p, TreeSegment& g) {
    if (at >= end) return false;
    while (in >= s.pieces(p.hkv)) {         // the next sequence with any
      if (++seq >= p.num_seqs) return false;
      in = 0;
      s = tree_seq(p, seq);
    }
    // (in 32 bits where that holds it: a 64-bit division takes hundreds of clocks)
    int64_t item;
    if (in <= 0xffffffffll) item = (uint32_t)in / (uint32_t)s.tiles;
    else item = in / s.tiles;
    g.seq = seq;
    g.unit = (int)item / p.hkv;
    g.head = (int)item - g.unit * p.hkv;
    g.t0 = (int)(in - item * s.tiles);
    g.t1 = (int)(end - at < s.tiles - g.t0 ? g.t0 + (end - at) : s.tiles);
    const bool whole = g.t0 == 0 && g.t1 == s.tiles;
    g.slot = whole ? -1 : 2 * cta + (at == begin ? 0 : 1);
    at += g.t1 - g.t0;
    in += g.t1 - g.t0;
    return true;
  }
};

// A (unit, head) that slice c continues and the slice before it began: the records
// of CTAs a = c - 1 to b, which the merge joins.  rows = 0: there is none.
struct __align__(16) TreeJoin {
  int q0, rows, head, slot_a;               // slot_a: of CTA a's record; the others' are 2 k
  int a, b, pad[2];
};

// By one thread of a CTA, behind the wait.  g: the walk's first segment (any: there is one).
__device__ __forceinline__ void tell_join(const TreePlan& p, const TreeWalk& walk, const TreeSegment& g, bool any, int64_t total) {
  TreeJoin j = {};
  if (any && g.t0 > 0) {
    const int c = walk.cta;
    const int64_t slices = tree_slices(p, total), begin = walk.begin - g.t0, before = tree_slice_begin(total, slices, c - 1);
    if (begin >= before) {
      const int tb = g.unit * p.unit_tokens;
      j.q0 = walk.s.q0 + tb;
      j.rows = min(p.unit_tokens, walk.s.n - tb) * p.group;
      j.head = g.head;
      j.slot_a = 2 * (c - 1) + (begin == before ? 0 : 1);
      j.a = c - 1;
      j.b = (int)tree_slice_of(total, slices, begin + walk.s.tiles - 1);
    }
  }
  p.join[walk.cta] = j;
}

}  // namespace pkvd
