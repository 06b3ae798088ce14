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
  // [num_seqs][max_q][words]: a node's visible ancestors and itself, a bit each;
  // by_key (at most 64 rows a tree): the rows of the nodes that see it, two words
  uint32_t* anc;
  int by_key;
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
  const bool ok = s.q0 >= 0 && s.n >= 0 && s.n <= p.max_q && s.cached >= 0 && (int64_t)s.q0 + s.n <= p.total_q &&
                  s.klen <= p.table_tokens;
  if (!ok) s.n = -1;
  if (s.n <= 0) return s;
  s.lo = p.window > 0 ? max(0, s.cached + 1 - p.window) : 0;
  s.lo_tile = s.lo / kTreeKeys;
  s.tiles = (s.klen - 1) / kTreeKeys - s.lo_tile + 1;
  s.units = (s.n + p.unit_tokens - 1) / p.unit_tokens;
  return s;
}

__device__ __forceinline__ TreeSeq tree_seq(const TreePlan& p, int i) {
  return tree_seq(p, p.cu_q[i], p.cu_q[i + 1] - p.cu_q[i], p.cu_k[i + 1] - p.cu_k[i]);
}

// Slices of a batch of `total` pieces, and where one begins.
__device__ __forceinline__ int64_t tree_slices(const TreePlan& p, int64_t total) {
  return total < p.grid ? total : p.grid;
}
__device__ __forceinline__ int64_t tree_slice_begin(int64_t total, int64_t slices, int64_t c) { return total * c / slices; }
// The slice that holds piece f.
__device__ __forceinline__ int64_t tree_slice_of(int64_t total, int64_t slices, int64_t f) {
  return ((f + 1) * slices - 1) / total;
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
  __device__ void start(const TreePlan& p, int c) {
    const TreeStart f = p.slice[c];
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

}  // namespace pkvd
