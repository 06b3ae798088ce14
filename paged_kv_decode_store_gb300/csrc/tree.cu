// Attention for trees of drafted tokens over the paged cache: the plan, the
// CUDA-core kernel and the merge; and the walk that says which drafts stay.
//
// Node t of sequence i's tree is its drafted row t, stored behind the cached
// tokens (position cached_i + t of the block table); parents[t] < t, or -1 for
// one that follows the cached context directly.  With depth(t) its ancestors'
// number, query head h of KV head hk = h / G:
//   out[t,h] = sum_j softmax_j(mod(scale <q[t,h], K_j>)) V_j
// over the cached keys (j < cached_i) and t's ancestors and t itself.  Token
// positions are cached_i + depth; a window and a distance bias count those.
//
// Parents become one bit a (node, ancestor) -- the window applied, so that a set
// bit is a visible key and the number of bits above one is its distance.  Three
// kernels compute the attention, chosen by type, layout and rows a tree (max_seqlen_q
// times the query heads of a KV head):
//   tree_few.cu, 16 bits, up to 64 rows: 32 sequences of 8 nodes, 48 + 8 heads of
//     128 over 2,048 tokens take 62 us (71 in tree_tc.cu; of 64 dims 51.5,
//     55.5 there; 24 sequences of up to 33 capped rows in a window 62, 64.5);
//   tree_tc.cu, 16 bits, more rows: up to 16 nodes there take 75 us;
//   below, fp32 and 16-bit caches whose layout the tensor copies cannot walk: four
//     sequences of up to 5 nodes in 15 us, as much as its launches.
// The last keeps 32 keys of K and V in shared memory and four query rows a warp:
// lane j scores key j, then owns D / 32 dims of the sums.  Bound by shared-memory
// reads (eight per sixteen multiply-adds).
#include "score_mod.cuh"
#include "tree_plan.cuh"

namespace pkvd {

cudaError_t launch_tree_tc(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream);    // tree_tc.cu
cudaError_t launch_tree_few(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream);   // tree_few.cu

namespace {

constexpr int kPlanThreads = 256, kNearSeqs = 1024;
static_assert(kPlanThreads >= kTreeMaxNodes, "a thread a node");

// A tree's visible ancestors, a bit each, and depths, by a CTA of a thread a node:
// what a thread leaves is its own node's (others read it behind a barrier).
__device__ __forceinline__ void tree_ancestors(const TreePlan& p, const int32_t* __restrict__ parents, const TreeSeq& s,
                                               uint32_t (*bits)[kTreeMaxNodes / 32 + 1], int* up, int* depths, int32_t* err) {
  const int tid = threadIdx.x;
  if (tid < s.n) {
    int u = parents[s.q0 + tid];
    if (u < -1 || u >= tid) {
      flag_error(err, PKVD_ERR_TREE);
      u = -1;
    }
    up[tid] = u;
  }
  for (int w = 0; w < p.words; ++w) bits[tid][w] = 0u;
  __syncthreads();
  if (tid >= s.n) return;
  int depth = -1;
  for (int u = tid; u >= 0; u = up[u]) {
    ++depth;
    if (p.window > 0 && depth >= p.window) continue;
    bits[tid][u >> 5] |= 1u << (u & 31);
  }
  depths[tid] = depth;
}

// CTA i < num_seqs: sequence i's ancestors.  The last one: the pieces before
// every sequence.  It runs where it is needed: for tree_tc.cu's masks, and for
// batches of more than kOwnSeqs sequences.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const TreePlan p, const int32_t* __restrict__ parents,
                                                                 int32_t* err) {
  __shared__ int up[kTreeMaxNodes], depths[kTreeMaxNodes];
  __shared__ uint32_t bits[kTreeMaxNodes][kTreeMaxNodes / 32 + 1];
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  __shared__ int64_t near[kNearSeqs];                // pieces before the first sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x == p.num_seqs) {
    // the lengths are inputs: summed up while the kernel before still runs (a call
    // before this one may still read the workspace: written behind the wait)
    const bool in_smem = p.num_seqs <= kNearSeqs;
    if (!in_smem) pdl_wait();
    int64_t running = 0;
    for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
      const int i = base + tid;
      const int64_t mine = i < p.num_seqs ? tree_seq(p, i).pieces(p.hkv) : 0;
      int64_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(FULL_MASK, upto, o);
        if (lane >= o) upto += t;
      }
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      int64_t before = running;
      for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        running += warp_sum[w];
      }
      if (i < p.num_seqs) (in_smem ? near : p.starts)[i] = before + upto - mine;
      __syncthreads();
    }
    // where the slices begin: in the last sequence with no more pieces before it
    const int64_t* starts = in_smem ? near : p.starts;
    const int64_t slices = tree_slices(p, running);
    auto begins = [&](int c) {
      const bool any = c < slices;
      const int64_t f = any ? tree_slice_begin(running, slices, c) : 0;
      int lo = 0, hi = p.num_seqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= f) lo = mid;
        else hi = mid;
      }
      TreeStart s;
      s.at = f;
      s.end = any ? tree_slice_begin(running, slices, c + 1) : 0;
      s.in = any ? f - starts[lo] : 0;
      s.seq = lo;
      s.q0 = p.cu_q[lo];
      s.n = p.cu_q[lo + 1] - s.q0;
      s.klen = p.cu_k[lo + 1] - p.cu_k[lo];
      s.pad[0] = s.pad[1] = 0;
      return s;
    };
    const TreeStart first = begins(tid);
    if (in_smem) pdl_wait();
    pdl_trigger();
    if (in_smem)
      for (int i = tid; i < p.num_seqs; i += kPlanThreads) p.starts[i] = near[i];
    if (tid == 0) p.starts[p.num_seqs] = running;
    if (tid < p.grid) p.slice[tid] = first;
    for (int c = tid + kPlanThreads; c < p.grid; c += kPlanThreads) p.slice[c] = begins(c);
    return;
  }
  const int i = blockIdx.x;
  const TreeSeq s = tree_seq(p, i);
  if (s.n < 0 && tid == 0) flag_error(err, PKVD_ERR_CONTEXT);
  tree_ancestors(p, parents, s, bits, up, depths, err);
  pdl_wait();
  pdl_trigger();
  if (tid < s.n) {
    const int64_t row = (int64_t)i * p.max_q + tid;
    p.depth[row] = depths[tid];
    for (int w = 0; w < p.words; ++w) p.anc[row * p.words + w] = bits[tid][w];
  }
}

// ------------------------------------------------------------- fp32 kernel
constexpr int kFmaThreads = 256, kFmaWarps = kFmaThreads / 32;
constexpr int kRowsPerWarp = 4, kPassRows = kFmaWarps * kRowsPerWarp;
constexpr int kChunkKeys = 32;

struct TreeFma {
  TreePlan plan;
  const int32_t* parents;
  void* out;
  const void* q;
  const uint8_t* kc;
  const uint8_t* vc;
  int64_t num_blocks, block_stride, token_stride, head_stride;   // strides in elements
  int block_size;
  const int32_t* tables;
  int max_blocks;
  float scale_log2;
  ScoreMod mod;
  int32_t* err;
};

// Is node u among the visible ancestors of a row, and how many lie after it?
__device__ __forceinline__ bool tree_sees(const uint32_t* anc, int words, int u, int& after) {
  const int w = u >> 5;
  const uint32_t x = anc[w];
  after = __popc(u % 32 == 31 ? 0u : x >> (u % 32 + 1));
  for (int k = w + 1; k < words; ++k) after += __popc(anc[k]);
  return (x >> (u & 31)) & 1u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kFmaThreads) tree_fma_kernel(const TreeFma p) {
  constexpr int LD = D + 4, DL = D / 32;
  extern __shared__ __align__(16) float sm[];
  float* ks = sm;                                   // [32][LD]
  float* vs = ks + kChunkKeys * LD;
  float* qs = vs + kChunkKeys * LD;                 // [kPassRows][D]
  float* ps = qs + kPassRows * D;                   // [kPassRows][32]
  uint32_t (*bits)[kTreeMaxNodes / 32 + 1] = reinterpret_cast<uint32_t (*)[kTreeMaxNodes / 32 + 1]>(ps + kPassRows * 32);
  int* up = reinterpret_cast<int*>(bits + kTreeMaxNodes);      // [kTreeMaxNodes]
  int* depths = up + kTreeMaxNodes;
  const TreePlan& pl = p.plan;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  TreeWalk walk;
  int64_t total;
  if (!pl.planned) {
    const OwnStart own(pl, blockIdx.x, lane);
    pdl_wait();
    pdl_trigger();
    walk.start(pl, blockIdx.x, own.first);
    total = own.total;
    if (own.bad && blockIdx.x == 0) flag_error(p.err, PKVD_ERR_CONTEXT);
  } else {
    pdl_wait();
    pdl_trigger();
    walk.start(pl, blockIdx.x, pl.slice[blockIdx.x]);
    total = pl.starts[pl.num_seqs];
  }
  TreeSegment g;
  int tree_of = -1;                                 // whose ancestors are at hand
  bool more = walk.next(pl, g);
  if (tid == 0) tell_join(pl, walk, g, more, total);
  for (; more; more = walk.next(pl, g)) {
    const TreeSeq& s = walk.s;
    if (g.seq != tree_of) {
      tree_of = g.seq;
      __syncthreads();
      tree_ancestors(pl, p.parents, s, bits, up, depths, p.err);
      __syncthreads();
    }
    const int tb = g.unit * pl.unit_tokens, rows = (min(tb + pl.unit_tokens, s.n) - tb) * pl.group;
    const int k0 = max(s.lo, (s.lo_tile + g.t0) * kTreeKeys), k1 = min(s.klen, (s.lo_tile + g.t1) * kTreeKeys);
    for (int pass = 0; pass < rows; pass += kPassRows) {
      float acc[kRowsPerWarp][DL], m[kRowsPerWarp], l[kRowsPerWarp], slope[kRowsPerWarp];
      int pos[kRowsPerWarp];
      const uint32_t* anc[kRowsPerWarp];
      __syncthreads();
      for (int idx = tid; idx < kPassRows * (D / 4); idx += kFmaThreads) {
        const int r = idx / (D / 4), c = idx % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (pass + r < rows) {
          const int t = (pass + r) / pl.group, gi = (pass + r) % pl.group;
          const T* src = static_cast<const T*>(p.q) +
                         ((int64_t)(s.q0 + tb + t) * pl.hq + (int64_t)g.head * pl.group + gi) * D + c;
          x = make_float4(DT<T>::to_f(src[0]), DT<T>::to_f(src[1]), DT<T>::to_f(src[2]), DT<T>::to_f(src[3]));
        }
        *reinterpret_cast<float4*>(qs + r * D + c) = x;
      }
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        const int row = min(pass + warp * kRowsPerWarp + r, rows - 1), t = row / pl.group;   // rows past the last mirror it
        pos[r] = s.cached + depths[tb + t];
        anc[r] = bits[tb + t];
        slope[r] = bias_slope(p.mod, g.head * pl.group + row % pl.group);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int d = 0; d < DL; ++d) acc[r][d] = 0.f;
      }
      for (int kb = k0; kb < k1; kb += kChunkKeys) {
        __syncthreads();
        for (int idx = tid; idx < kChunkKeys * (D / 4); idx += kFmaThreads) {
          const int r = idx / (D / 4), c = idx % (D / 4) * 4, j = kb + r;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
          if (j < k1) {
            const int b = __ldg(p.tables + (int64_t)g.seq * p.max_blocks + j / p.block_size);
            if (b >= 0 && b < p.num_blocks) {
              const int64_t off = (int64_t)b * p.block_stride + (int64_t)(j % p.block_size) * p.token_stride +
                                  (int64_t)g.head * p.head_stride + c;
              const T* kp = reinterpret_cast<const T*>(p.kc) + off;
              const T* vp = reinterpret_cast<const T*>(p.vc) + off;
              x = make_float4(DT<T>::to_f(kp[0]), DT<T>::to_f(kp[1]), DT<T>::to_f(kp[2]), DT<T>::to_f(kp[3]));
              y = make_float4(DT<T>::to_f(vp[0]), DT<T>::to_f(vp[1]), DT<T>::to_f(vp[2]), DT<T>::to_f(vp[3]));
            } else if (c == 0) {
              flag_error(p.err, PKVD_ERR_BLOCK_ID);              // its keys read as zeros
            }
          }
          *reinterpret_cast<float4*>(ks + r * LD + c) = x;
          *reinterpret_cast<float4*>(vs + r * LD + c) = y;
        }
        __syncthreads();
        if (pass + warp * kRowsPerWarp >= rows) continue;
        float sc[kRowsPerWarp] = {};
        const float* qw = qs + warp * kRowsPerWarp * D;
#pragma unroll 8
        for (int c = 0; c < D; c += 4) {
          const float4 k = *reinterpret_cast<const float4*>(ks + lane * LD + c);
#pragma unroll
          for (int r = 0; r < kRowsPerWarp; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(qw + r * D + c);
            sc[r] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, sc[r]))));
          }
        }
        const int j = kb + lane;
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
          int back = pos[r] - j;
          bool sees = j < k1 && (pl.window <= 0 || back < pl.window);
          if (j >= s.cached && j < k1) sees = tree_sees(anc[r], pl.words, j - s.cached, back);
          float x = -INFINITY;
          if (sees) x = fmaf(slope[r], (float)back, capped<std::is_same<T, float>::value>(sc[r], p.scale_log2, p.mod));
          float top = x;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
          const float mn = fmaxf(m[r], top), base = mn == -INFINITY ? 0.f : mn;
          const float corr = exp2f(m[r] - base), e = exp2f(x - base);
          float sum = e;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
          l[r] = l[r] * corr + sum;
          m[r] = mn;
#pragma unroll
          for (int d = 0; d < DL; ++d) acc[r][d] *= corr;
          ps[(warp * kRowsPerWarp + r) * 32 + lane] = e;
        }
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < kChunkKeys; k += 4) {
          float4 w[kRowsPerWarp];
#pragma unroll
          for (int r = 0; r < kRowsPerWarp; ++r)
            w[r] = *reinterpret_cast<const float4*>(ps + (warp * kRowsPerWarp + r) * 32 + k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v[DL];
#pragma unroll
            for (int d = 0; d < DL; ++d) v[d] = vs[(k + e) * LD + lane * DL + d];
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r) {
              const float x = e == 0 ? w[r].x : e == 1 ? w[r].y : e == 2 ? w[r].z : w[r].w;
              // a key that this row does not see weighs nothing, whatever its value holds
#pragma unroll
              for (int d = 0; d < DL; ++d) acc[r][d] = x == 0.f ? acc[r][d] : fmaf(x, v[d], acc[r][d]);
            }
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        const int row = pass + warp * kRowsPerWarp + r;
        if (row >= rows) continue;
        if (g.slot < 0) {
          const int t = row / pl.group, gi = row % pl.group;
          T* dst = static_cast<T*>(p.out) + ((int64_t)(s.q0 + tb + t) * pl.hq + (int64_t)g.head * pl.group + gi) * D;
          const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
          for (int d = 0; d < DL; ++d) dst[lane * DL + d] = DT<T>::from_f(acc[r][d] * inv);
        } else {
          const int64_t at = (int64_t)g.slot * pl.unit_rows + row;
#pragma unroll
          for (int d = 0; d < DL; ++d) pl.rec[at * D + lane * DL + d] = acc[r][d];
          if (lane == 0) pl.rec_ml[at] = make_float2(m[r], l[r]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------- merge
// Joins the records of a (unit, head) that more than one CTA worked on:
//   M = max m_k, out = sum 2^(m_k - M) acc_k / sum 2^(m_k - M) l_k.
// CTA (c, group): what slice c continues and the one before began, as CTA c of the
// kernel with the records left it (finding it here, for every unit of every
// sequence, took divisions by every CTA: 312 instead of 308 us for 16 sequences of 64
// nodes of 64 heads).
// PARTS = 1: a warp has kMergeRows rows, whose records are on their way together
// (one row a warp: 36 instead of 18 us for 64 nodes of 8 heads a KV head, where
// rows are cut in two or three).  PARTS = 8, for few rows cut into many pieces:
// the CTA's eight warps share a row's records.
constexpr int kMergeRows = 4;

template <typename T, int D, int PARTS>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreePlan p, T* __restrict__ out) {
  constexpr int ROWS = PARTS == 1 ? kMergeRows : 1, R = PARTS == 1 ? 3 : 8;   // rows, records of each on their way
  __shared__ float part[PARTS == 1 ? 1 : 8 * (D + 2)];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = blockIdx.y;
  int c = blockIdx.x;
  if constexpr (PARTS > 1) {           // few of the slices' begins have something to join: the x-th of those
    int left = blockIdx.x;
    c = -1;
#pragma unroll 4
    for (int base = 0; base < p.grid; base += 32) {
      const uint32_t some = __ballot_sync(FULL_MASK, base + lane < p.grid && p.join[base + lane].rows > 0);
      const int n = __popc(some);
      if (c < 0 && left < n) c = base + __fns(some, 0, left + 1);
      left -= n;
    }
    if (c < 0) return;
  }
  const TreeJoin j = p.join[c];
  const int rows = j.rows, a = j.a, b = j.b;
  const int row0 = PARTS == 1 ? (group * 8 + warp) * ROWS : group;
  if ((PARTS == 1 ? group * 8 * ROWS : group) >= rows) return;
  constexpr int Q = D / 4, SUB = 32 / Q;                 // lanes of a row's float4 slices; records a warp takes at once
  const int d4 = lane % Q * 4, sub = lane / Q;
  const int step = SUB * PARTS, k_first = PARTS == 1 ? sub : warp * SUB + sub;
  float M[ROWS], L[ROWS];
  float4 o[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) M[i] = -INFINITY, L[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = a + k_first; row0 < rows && k0 <= b; k0 += R * step) {
    float2 ml[R][ROWS];
    float4 x[R][ROWS];
#pragma unroll
    for (int e = 0; e < R; ++e) {
      const int k = k0 + e * step;
      const int64_t at = (int64_t)(k == a ? j.slot_a : 2 * k) * p.unit_rows + row0;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        ml[e][i] = make_float2(-INFINITY, 0.f);
        x[e][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= b && row0 + i < rows) {
          ml[e][i] = p.rec_ml[at + i];
          x[e][i] = *reinterpret_cast<const float4*>(p.rec + (at + i) * D + d4);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < R; ++e)
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        // saw none of the keys (where all that it saw were NaN the sum is one, and no maximum was found either)
        if (ml[e][i].y == 0.f) continue;
        const float Mn = fmaxf(M[i], ml[e][i].x), cs = exp2f(M[i] - Mn), cr = exp2f(ml[e][i].x - Mn);
        L[i] = L[i] * cs + ml[e][i].y * cr;
        o[i].x = o[i].x * cs + x[e][i].x * cr;
        o[i].y = o[i].y * cs + x[e][i].y * cr;
        o[i].z = o[i].z * cs + x[e][i].z * cr;
        o[i].w = o[i].w * cs + x[e][i].w * cr;
        M[i] = Mn;
      }
  }
  auto join = [&](int i, float Mo, float Lo, float4 x) {
    const float Mn = fmaxf(M[i], Mo), base = Mn == -INFINITY ? 0.f : Mn;
    const float ca = exp2f(M[i] - base), cb = exp2f(Mo - base);
    L[i] = L[i] * ca + Lo * cb;
    o[i] = make_float4(o[i].x * ca + x.x * cb, o[i].y * ca + x.y * cb, o[i].z * ca + x.z * cb, o[i].w * ca + x.w * cb);
    M[i] = Mn;
  };
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int off = Q; off < 32; off <<= 1) {
      const float Mo = __shfl_xor_sync(FULL_MASK, M[i], off), Lo = __shfl_xor_sync(FULL_MASK, L[i], off);
      const float4 x = make_float4(__shfl_xor_sync(FULL_MASK, o[i].x, off), __shfl_xor_sync(FULL_MASK, o[i].y, off),
                                   __shfl_xor_sync(FULL_MASK, o[i].z, off), __shfl_xor_sync(FULL_MASK, o[i].w, off));
      join(i, Mo, Lo, x);
    }
  if constexpr (PARTS > 1) {
    float* mine = part + warp * (D + 2);
    if (sub == 0) {
      mine[d4] = o[0].x, mine[d4 + 1] = o[0].y, mine[d4 + 2] = o[0].z, mine[d4 + 3] = o[0].w;
      if (d4 == 0) mine[D] = M[0], mine[D + 1] = L[0];
    }
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < 8; ++w) {
      const float* x = part + w * (D + 2);
      join(0, x[D], x[D + 1], make_float4(x[d4], x[d4 + 1], x[d4 + 2], x[d4 + 3]));
    }
  }
  if (sub > 0) return;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i;
    if (row >= rows) break;
    const int t = row / p.group, gi = row % p.group;
    T* dst = out + ((int64_t)(j.q0 + t) * p.hq + (int64_t)j.head * p.group + gi) * D + d4;
    const float inv = L[i] > 0.f ? 1.f / L[i] : 0.f;
    if constexpr (sizeof(T) == 2) {                      // out is 16-byte aligned, rows of 128 bytes and more
      *reinterpret_cast<uint2*>(dst) = make_uint2(Mma<T>::pack(o[i].x * inv, o[i].y * inv), Mma<T>::pack(o[i].z * inv, o[i].w * inv));
    } else {
      *reinterpret_cast<float4*>(dst) = make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
    }
  }
}

// ------------------------------------------------------------------ accept
// A warp a sequence.  Node 0 is the token that the target chose last; from a
// node on the path the walk goes to the lowest child that drafts the target's
// choice there, eight nodes a lane in registers.
constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const AcceptArgs a, int num_seqs) {
  constexpr int PER = kTreeMaxNodes / 32;
  pdl_wait();          // the target's choices come from the sampler (no early trigger: counts may be lengths)
  const int i = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= num_seqs) return;
  const int q0 = a.cu_q[i], n = a.cu_q[i + 1] - q0, klen = a.cu_k[i + 1] - a.cu_k[i], cached = klen - n;
  int count = 0;
  const bool ok = q0 >= 0 && n >= 0 && n <= kTreeMaxNodes && klen >= n && (int64_t)q0 + n <= a.total_q;
  if (!ok && lane == 0) flag_error(a.err, PKVD_ERR_CONTEXT);
  int32_t* pos = a.positions + (int64_t)i * a.max_path;
  int32_t* tok = a.tokens + (int64_t)i * a.max_path;
  if (ok && n > 0) {
    int up[PER], id[PER], choice[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int t = k * 32 + lane;
      up[k] = id[k] = choice[k] = -1;
      if (t < n) {
        up[k] = a.parents[q0 + t];
        id[k] = a.drafted[q0 + t];
        choice[k] = a.target[q0 + t];
        if (up[k] < -1 || up[k] >= t) {
          flag_error(a.err, PKVD_ERR_TREE);
          up[k] = -1;
        }
      }
    }
    int here = 0;
    while (count < a.max_path) {
      int want = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = __shfl_sync(FULL_MASK, choice[k], here & 31);
        if (k == here >> 5) want = c;
      }
      if (lane == 0) {
        pos[count] = cached + here;
        tok[count] = want;
      }
      ++count;
      int child = -1;
#pragma unroll
      for (int k = PER - 1; k >= 0; --k) {
        const uint32_t fits = __ballot_sync(FULL_MASK, up[k] == here && id[k] == want && k * 32 + lane < n);
        if (fits) child = k * 32 + __ffs(fits) - 1;
      }
      if (child < 0) break;
      here = child;
    }
  }
  for (int k = count + lane; k < a.max_path; k += 32) pos[k] = tok[k] = -1;
  if (lane == 0) {
    a.first[i] = ok ? cached : 0;
    a.counts[i] = count;
    __threadfence();
  }
}

// ------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int words_of(int max_q) { return (max_q + 31) / 32; }

bool few_rows(int group, int max_q) { return group * max_q <= kTreeFewRows; }

int unit_tokens_of(int path, int group, int max_q) {
  if (path == PKVD_PATH_FMA) return kPassRows / group > 1 ? kPassRows / group : 1;
  // trees of few rows: a unit is a whole tree, its rows the columns of tree_few.cu
  if (few_rows(group, max_q)) return max_q;
  const int tile = 128 / group;                          // two Q tiles, or one where that holds every tree
  return max_q > tile ? 2 * tile : tile;
}

int grid_of(int path, int sms) { return path == PKVD_PATH_FMA ? 2 * sms : sms; }

struct WorkspaceLayout {
  size_t starts, slice, join, anc, depth, rec, rec_ml, bytes;
  WorkspaceLayout(int path, int num_seqs, int group, int head_dim, int max_q, int sms) {
    const int words = words_of(max_q);
    const size_t rows = (size_t)2 * grid_of(path, sms) * unit_tokens_of(path, group, max_q) * group;
    starts = 0;
    slice = starts + up256(sizeof(int64_t) * ((size_t)num_seqs + 1));
    join = slice + up256(sizeof(TreeStart) * (size_t)grid_of(path, sms));
    anc = join + up256(sizeof(TreeJoin) * (size_t)grid_of(path, sms));
    depth = anc + up256(sizeof(uint32_t) * (size_t)num_seqs * max_q * words);
    rec_ml = depth + up256(sizeof(int32_t) * (size_t)num_seqs * max_q);
    rec = rec_ml + up256(sizeof(float2) * rows);
    bytes = rec + up256(sizeof(float) * rows * head_dim);
  }
};

template <typename T, int D>
cudaError_t launch_fma(const TreeFma& p, cudaStream_t stream) {
  constexpr int smem = (2 * kChunkKeys * (D + 4) + kPassRows * (D + 32) + kTreeMaxNodes * (kTreeMaxNodes / 32 + 3)) * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(tree_fma_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_fma_kernel<T, D>, dim3(p.plan.grid), dim3(kFmaThreads), smem, stream, p);
}

template <typename T, int D>
cudaError_t launch_merge(const TreePlan& p, void* out, cudaStream_t stream) {
  const int64_t items = (int64_t)((p.max_q + p.unit_tokens - 1) / p.unit_tokens) * p.hkv;
  const int rows = (p.max_q < p.unit_tokens ? p.max_q : p.unit_tokens) * p.group;
  // pieces of an item: about grid / items; a warp takes eight records a round
  const bool many = p.grid > 8 * items * p.num_seqs;
  const dim3 grid((unsigned)(many ? items * p.num_seqs : p.grid), (unsigned)(many ? rows : (rows + 8 * kMergeRows - 1) / (8 * kMergeRows)));
  return many ? launch_pdl(tree_merge_kernel<T, D, 8>, grid, dim3(256), 0, stream, p, static_cast<T*>(out))
              : launch_pdl(tree_merge_kernel<T, D, 1>, grid, dim3(256), 0, stream, p, static_cast<T*>(out));
}

}  // namespace

// Enough for either path: a call whose layout the tensor cores cannot read falls back.
size_t tree_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_seqlen_q, int sms) {
  const int group = num_q_heads / num_kv_heads;
  const size_t a = WorkspaceLayout(PKVD_PATH_FMA, num_seqs, group, head_dim, max_seqlen_q, sms).bytes;
  const size_t b = WorkspaceLayout(PKVD_PATH_TC, num_seqs, group, head_dim, max_seqlen_q, sms).bytes;
  return a > b ? a : b;
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const pkvd_cache& c = a.cache;
  const int group = a.num_q_heads / c.num_kv_heads;
  const WorkspaceLayout lay(a.path, a.num_seqs, group, c.head_dim, a.max_seqlen_q, a.sms);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  TreePlan p;
  p.cu_q = a.cu_seqlens_q;
  p.cu_k = a.cu_seqlens_k;
  p.num_seqs = a.num_seqs;
  p.total_q = a.total_q;
  p.max_q = a.max_seqlen_q;
  p.words = words_of(a.max_seqlen_q);
  p.unit_tokens = unit_tokens_of(a.path, group, a.max_seqlen_q);
  p.unit_rows = p.unit_tokens * group;
  p.hkv = c.num_kv_heads;
  p.hq = a.num_q_heads;
  p.group = group;
  p.window = a.window;
  p.table_tokens = (int64_t)a.max_blocks_per_seq * c.block_size;
  p.grid = grid_of(a.path, a.sms);
  p.planned = a.num_seqs > kOwnSeqs || (a.path == PKVD_PATH_TC && !few_rows(group, a.max_seqlen_q));
  p.starts = reinterpret_cast<int64_t*>(ws + lay.starts);
  p.slice = reinterpret_cast<TreeStart*>(ws + lay.slice);
  p.join = reinterpret_cast<TreeJoin*>(ws + lay.join);
  p.anc = reinterpret_cast<uint32_t*>(ws + lay.anc);
  p.depth = reinterpret_cast<int32_t*>(ws + lay.depth);
  p.rec = reinterpret_cast<float*>(ws + lay.rec);
  p.rec_ml = reinterpret_cast<float2*>(ws + lay.rec_ml);
  cudaError_t e = cudaSuccess;
  if (p.planned) e = launch_pdl(tree_plan_kernel, dim3(a.num_seqs + 1), dim3(kPlanThreads), 0, stream, p, a.parents, a.err);
  if (e != cudaSuccess) return e;
  if (a.path == PKVD_PATH_TC) {
    e = few_rows(group, a.max_seqlen_q) ? launch_tree_few(a, p, stream) : launch_tree_tc(a, p, stream);
  } else {
    TreeFma f;
    f.plan = p;
    f.parents = a.parents;
    f.out = a.out;
    f.q = a.q;
    f.kc = static_cast<const uint8_t*>(c.k_base);
    f.vc = static_cast<const uint8_t*>(c.v_base);
    f.num_blocks = c.num_blocks;
    f.block_stride = c.block_stride;
    f.token_stride = c.token_stride;
    f.head_stride = c.head_stride;
    f.block_size = c.block_size;
    f.tables = a.block_tables;
    f.max_blocks = a.max_blocks_per_seq;
    f.scale_log2 = a.scale * 1.4426950408889634f;
    f.mod = a.mod;
    f.err = a.err;
    const bool wide = c.head_dim == 128;
    if (c.dtype == PKVD_F32) e = wide ? launch_fma<float, 128>(f, stream) : launch_fma<float, 64>(f, stream);
    else if (c.dtype == PKVD_F16) e = wide ? launch_fma<__half, 128>(f, stream) : launch_fma<__half, 64>(f, stream);
    else e = wide ? launch_fma<__nv_bfloat16, 128>(f, stream) : launch_fma<__nv_bfloat16, 64>(f, stream);
  }
  if (e != cudaSuccess) return e;
  if (p.table_tokens <= kTreeKeys) return cudaSuccess;     // a tile of keys each: nothing is cut
  const bool wide = c.head_dim == 128;
  if (c.dtype == PKVD_F32) return wide ? launch_merge<float, 128>(p, a.out, stream) : launch_merge<float, 64>(p, a.out, stream);
  if (c.dtype == PKVD_F16) return wide ? launch_merge<__half, 128>(p, a.out, stream) : launch_merge<__half, 64>(p, a.out, stream);
  return wide ? launch_merge<__nv_bfloat16, 128>(p, a.out, stream) : launch_merge<__nv_bfloat16, 64>(p, a.out, stream);
}

cudaError_t launch_tree_accept(const AcceptArgs& a, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0) return cudaSuccess;
  return launch_pdl(tree_accept_kernel, dim3((num_seqs + kAcceptWarps - 1) / kAcceptWarps), dim3(kAcceptWarps * 32), 0,
                    stream, a, num_seqs);
}

}  // namespace pkvd
