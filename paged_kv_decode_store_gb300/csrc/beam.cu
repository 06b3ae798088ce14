// One step of beam search: of all continuations (beam b, id j) of a request,
// the `keep` with the largest
//   scores[b] + x_bj - logsumexp_j(x_bj),
// the lowest b * vocab + j first among equal values.
//
// Two kernels.  The scan reads every logit once: a row is cut into slices of
// 32 KB, one CTA each, held in registers (four 16-byte loads a thread, all in
// flight together).  From one pass come the slice's maximum, its sum of
// exponentials and its `keep` best ids -- enough, since a request's best
// `keep` continuations are among the best `keep` of their slices.  They are
// found without sorting: the maxima of 64 disjoint groups of the slice are
// `keep` or more distinct elements, so the keep-th largest group maximum is a
// lower bound of the keep-th largest element; the few elements at or above it
// are listed and ranked against one another.  The merge, one CTA per request,
// joins the slices' sums into each beam's normaliser and selects the same way
// among the slices' candidates.
//
// Rounding: within a beam the order is that of the logits themselves (exact);
// between beams the values are compared in 64 bits: the normaliser's sum is
// fp32 within a slice (32 terms a thread, then a tree: about 2^-24 relative),
// joined and turned into a logarithm in fp64.
//
// Bound: the logits' bytes for large batches; for small ones the two
// kernels' latency.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kBeamThreads = 512;
constexpr int kBeamVecs = 4;                          // 16-byte vectors a thread holds
constexpr int kSliceVecs = kBeamThreads * kBeamVecs;  // 16-byte vectors of a slice
constexpr int kGroups = 64;                           // groups of 8 lanes: kBeamMaxKeep of them
constexpr int kBeamList = 2048;                       // listed elements; more take the slow selection
static_assert(kGroups >= kBeamMaxKeep && kBeamThreads == kGroups * 8, "a bound needs keep groups");

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Float bits in an order-preserving unsigned form; 0 is below every number.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered(uint64_t k) {
  return __longlong_as_double((long long)(k ^ ((k >> 63) ? 1ull << 63 : ~0ull)));
}

// The keep-th largest of the kGroups values in s_group (called by kGroups
// threads; the one that holds it returns true).
template <typename V>
__device__ __forceinline__ bool is_kth(const V* s_group, int t, int keep) {
  const V v = s_group[t];
  int before = 0;
#pragma unroll 16
  for (int j = 0; j < kGroups; ++j) before += s_group[j] > v || (s_group[j] == v && j < t);
  return before == keep - 1;
}

struct ScanSmem {
  float warp_max[kBeamThreads / 32];
  float warp_sum[kBeamThreads / 32];
  float group[kGroups];
  float bound;
  int count;
  uint64_t best;
  uint64_t list[kBeamList];
};

// A candidate of a slice: the logit's ordered bits, then the lower id first.
__device__ __forceinline__ uint64_t cand(float x, int id) {
  return ((uint64_t)ordered(x + 0.f) << 32) | (0xffffffffu - (uint32_t)id);   // -0 counts as 0
}

template <typename T>
__global__ void __launch_bounds__(kBeamThreads) beam_scan_kernel(const BeamArgs p) {
  constexpr int N = Vec16<T>::N;
  __shared__ ScanSmem s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  pdl_wait();
  pdl_trigger();
  if (p.finished && p.finished[row]) return;           // an ended beam: its logits do not count
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.row_stride;
  // the row from the 16-byte boundary at or before it: element e of that is id e - lead
  const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const T* base = x - lead;
  const int end = lead + p.vocab;
  float v[kBeamVecs][N];
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < kBeamVecs; ++i) {
    const int64_t e0 = ((int64_t)split * kSliceVecs + i * kBeamThreads + tid) * N;
    const bool whole = e0 >= lead && e0 + N <= end;
    const uint4 raw = whole ? __ldg(reinterpret_cast<const uint4*>(base + e0)) : none;
    Vec16<T>::unpack(raw, v[i]);
    if (!whole) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = e0 + j >= lead && e0 + j < end ? DT<T>::to_f(base[e0 + j]) : -INFINITY;
    }
  }
  if (tid == 0) s.count = 0;
  float most = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBeamVecs; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) most = fmaxf(most, v[i][j]);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, o));
  if ((lane & 7) == 0) s.group[tid >> 3] = most;
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, o));
  if (lane == 0) s.warp_max[warp] = most;
  __syncthreads();
  if (tid < kGroups && is_kth(s.group, tid, p.keep)) s.bound = s.group[tid];
  float m = s.warp_max[lane & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
  // a NaN or +inf logit makes the sum NaN: the merge then drops the beam
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kBeamVecs; ++i) {
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) part += ex2f((v[i][j] - ref) * 1.4426950408889634f);
    sum += part;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
  if (lane == 0) s.warp_sum[warp] = sum;
  __syncthreads();
  const float bound = s.bound;
#pragma unroll
  for (int i = 0; i < kBeamVecs; ++i) {
    const int id0 = (int)(((int64_t)split * kSliceVecs + i * kBeamThreads + tid) * N) - lead;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (v[i][j] >= bound && v[i][j] > -INFINITY) {
        const int at = atomicAdd(&s.count, 1);
        if (at < kBeamList) s.list[at] = cand(v[i][j], id0 + j);
      }
    }
  }
  __syncthreads();
  const int64_t slice = (int64_t)row * p.splits + split;
  uint64_t* out = p.cands + slice * p.keep;
  const int n = s.count;
  if (tid == 0) {
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kBeamThreads / 32; ++w) total += s.warp_sum[w];
    p.sums[slice] = make_float2(m, total);
  }
  if (n <= kBeamList) {
    for (int i = tid; i < n; i += kBeamThreads) {
      const uint64_t mine = s.list[i];
      int before = 0;
      for (int j = 0; j < n; ++j) before += s.list[j] > mine;          // no two are equal
      if (before < p.keep) out[before] = mine;
    }
    for (int i = n + tid; i < p.keep; i += kBeamThreads) out[i] = 0;
  } else {
    // so many equal to the bound: the best one below the last, keep times
    uint64_t last = ~0ull;
    for (int k = 0; k < p.keep; ++k) {
      if (tid == 0) s.best = 0;
      __syncthreads();
      uint64_t mine = 0;
#pragma unroll
      for (int i = 0; i < kBeamVecs; ++i) {
        const int id0 = (int)(((int64_t)split * kSliceVecs + i * kBeamThreads + tid) * N) - lead;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint64_t c = v[i][j] > -INFINITY ? cand(v[i][j], id0 + j) : 0;
          if (c < last && c > mine) mine = c;
        }
      }
      atomicMax(reinterpret_cast<unsigned long long*>(&s.best), (unsigned long long)mine);
      __syncthreads();
      last = s.best;
      if (tid == 0) out[k] = last;
      __syncthreads();
    }
  }
}

struct MergeSmem {
  double base[kBeamMaxBeams];            // score minus normaliser, -inf: the beam offers nothing
  uint64_t group[kGroups];
  uint64_t bound;
  int count;
  unsigned long long best;
  uint32_t best_at;
  uint64_t value[kBeamList];
  uint32_t at[kBeamList];
};

// One CTA per request.
__global__ void __launch_bounds__(kBeamThreads) beam_merge_kernel(const BeamArgs p) {
  __shared__ MergeSmem s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x, B = p.beams, K = p.keep;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) s.count = 0;
  // each beam's normaliser: a warp per beam over its slices
  for (int b = warp; b < B; b += kBeamThreads / 32) {
    const int row = r * B + b;
    const double score = (double)p.scores[row];
    double base = score;
    const bool ended = p.finished && p.finished[row];
    if (!ended) {
      const float2* part = p.sums + (int64_t)row * p.splits;
      float m = -INFINITY;
      bool bad = false;
      for (int i = lane; i < p.splits; i += 32) {
        const float2 t = part[i];
        m = fmaxf(m, t.x);
        bad |= !(t.y < INFINITY);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
      double total = 0.0;
      for (int i = lane; i < p.splits; i += 32) {
        const float2 t = part[i];
        if (t.y > 0.f) total += (double)t.y * exp((double)t.x - (double)m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL_MASK, total, o);
      bad = __any_sync(FULL_MASK, bad);
      base = bad || !(total > 0.0) ? -INFINITY : score - ((double)m + log(total));
    }
    if (lane == 0) s.base[b] = base > -INFINITY && base < INFINITY ? base : -INFINITY;
  }
  __syncthreads();
  // candidate c: the k-th best of a slice of a beam, or an ended beam's own
  // continuation; value 0 (below every number) if it is none
  const int per = p.splits * K;
  const int64_t nc = (int64_t)B * per + B;
  auto candidate = [&](int64_t c, uint64_t& value, uint32_t& at) {
    value = 0;
    at = 0;
    const bool own = c >= (int64_t)B * per;
    const int b = own ? (int)(c - (int64_t)B * per) : (int)(c / per);
    const double base = s.base[b];
    if (base == -INFINITY) return;
    const bool ended = p.finished && p.finished[r * B + b];
    if (own != ended) return;
    if (own) {
      value = ordered(base);
      at = (uint32_t)b * p.vocab + p.eos_id;
      return;
    }
    const uint64_t key = p.cands[(int64_t)(r * B + b) * per + (c - (int64_t)b * per)];
    if (key == 0) return;
    value = ordered(base + (double)unordered((uint32_t)(key >> 32)) + 0.0);
    at = (uint32_t)b * p.vocab + (0xffffffffu - (uint32_t)key);
  };
  uint64_t most = 0;
  for (int64_t c = tid; c < nc; c += kBeamThreads) {
    uint64_t value;
    uint32_t at;
    candidate(c, value, at);
    most = value > most ? value : most;
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const uint64_t other = __shfl_xor_sync(FULL_MASK, most, o);
    most = other > most ? other : most;
  }
  if ((lane & 7) == 0) s.group[tid >> 3] = most;
  __syncthreads();
  if (tid < kGroups && is_kth(s.group, tid, K)) s.bound = s.group[tid];
  __syncthreads();
  const uint64_t bound = s.bound;
  for (int64_t c = tid; c < nc; c += kBeamThreads) {
    uint64_t value;
    uint32_t at;
    candidate(c, value, at);
    if (value != 0 && value >= bound) {
      const int i = atomicAdd(&s.count, 1);
      if (i < kBeamList) {
        s.value[i] = value;
        s.at[i] = at;
      }
    }
  }
  __syncthreads();
  auto emit = [&](int k, uint64_t value, uint32_t at) {
    const int64_t o = (int64_t)r * K + k;
    p.out_scores[o] = value ? (float)unordered(value) : -INFINITY;
    p.out_parents[o] = value ? (int)(at / (uint32_t)p.vocab) : -1;
    p.out_tokens[o] = value ? (int)(at % (uint32_t)p.vocab) : -1;
  };
  const int n = s.count;
  if (n <= kBeamList) {
    for (int i = tid; i < n; i += kBeamThreads) {
      const uint64_t value = s.value[i];
      const uint32_t at = s.at[i];
      int before = 0;
      for (int j = 0; j < n; ++j) before += s.value[j] > value || (s.value[j] == value && s.at[j] < at);
      if (before < K) emit(before, value, at);
    }
    for (int i = n + tid; i < K; i += kBeamThreads) emit(i, 0, 0);
  } else {
    uint64_t last = ~0ull;
    uint32_t last_at = 0;
    for (int k = 0; k < K; ++k) {
      if (tid == 0) {
        s.best = 0;
        s.best_at = 0xffffffffu;
      }
      __syncthreads();
      uint64_t mine = 0;
      uint32_t mine_at = 0xffffffffu;
      for (int64_t c = tid; c < nc; c += kBeamThreads) {
        uint64_t value;
        uint32_t at;
        candidate(c, value, at);
        const bool below = value < last || (value == last && at > last_at);
        if (value && below && (value > mine || (value == mine && at < mine_at))) mine = value, mine_at = at;
      }
      atomicMax(&s.best, (unsigned long long)mine);
      __syncthreads();
      if (mine && mine == s.best) atomicMin(&s.best_at, mine_at);
      __syncthreads();
      last = s.best;
      last_at = s.best_at;
      if (tid == 0) emit(k, last, last_at);
      __syncthreads();
      if (last == 0) {                                   // nothing left: the rest is empty
        for (int i = k + 1 + tid; i < K; i += kBeamThreads) emit(i, 0, 0);
        break;
      }
    }
  }
}

template <typename T>
cudaError_t launch_typed(const BeamArgs& a, cudaStream_t stream) {
  const int64_t ctas = (int64_t)a.requests * a.beams * a.splits;
  cudaError_t e = launch_pdl(beam_scan_kernel<T>, dim3((unsigned)ctas), dim3(kBeamThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_merge_kernel, dim3((unsigned)a.requests), dim3(kBeamThreads), 0, stream, a);
}

}  // namespace

// Slices of a row, whatever its alignment (a row may start inside its first vector).
int beam_splits(int dtype, int vocab) {
  const int n = dtype == PKVD_F32 ? 4 : 8;
  const int64_t vecs = ((int64_t)vocab + n - 1 + n - 1) / n;
  return (int)((vecs + kSliceVecs - 1) / kSliceVecs);
}

size_t beam_workspace_bytes(int64_t rows, int splits, int keep) {
  return (size_t)rows * splits * ((size_t)keep * sizeof(uint64_t) + sizeof(float2));
}

cudaError_t launch_beam(const BeamArgs& a, cudaStream_t stream) {
  if (a.dtype == PKVD_F32) return launch_typed<float>(a, stream);
  if (a.dtype == PKVD_F16) return launch_typed<__half>(a, stream);
  return launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace pkvd
