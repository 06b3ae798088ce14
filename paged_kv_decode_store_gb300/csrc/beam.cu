// One step of beam search: of all continuations (beam b, id j) of a request,
// the `keep` with the largest
//   scores[b] + x_bj - logsumexp_j(x_bj),
// the lowest b * vocab + j first among equal values.
//
// Two kernels.  The scan reads every logit once and selects nothing: a warp
// takes a span of 1 KB chunks (two 16-byte loads a lane each, the next two
// chunks in flight while two are summed) and leaves the span's maximum and sum
// of exponentials and each chunk's maximum -- no barrier, no shared memory.
// The merge, one CTA per request, joins the sums into each beam's normaliser
// and finds the winners from the maxima: the maxima of `keep` chunks are
// `keep` elements, so the keep-th largest chunk maximum bounds the keep-th
// best value from below, and only the few chunks that reach it are read again
// (from L2 or DRAM, a few KB).  The same argument on the vectors of those
// chunks tightens the bound; what is left (some more than `keep` elements) is
// listed and ranked against one another.
//
// Rounding: within a beam the order is that of the logits themselves (exact);
// between beams listed values are compared in 64 bits.  The bounds are fp32
// with a margin for their own rounding.  The normaliser's sum is fp32 within
// a span (16 terms at a time, then up to 16 such sums, then a tree: about
// 2^-24 relative), its logarithm fp64.
//
// Bound: the logits' bytes for large batches; for small ones the two
// kernels' latency.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pkvd {

namespace {

constexpr int kScanThreads = 256;                     // eight warps, each on its own
constexpr int kChunkVecs = 64;                        // 16-byte vectors of a chunk
constexpr int kMaxSpan = 16;                          // chunks a warp takes at most
constexpr int kMergeThreads = 512;
constexpr int kGroups = 64;                           // groups of 8 lanes of the merge
constexpr int kBeamList = 2048;                       // listed elements and chunks
static_assert(kGroups >= kBeamMaxKeep && kMergeThreads == kGroups * 8, "a bound needs keep groups");

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
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

// Where a row's vectors lie: from the 16-byte boundary at or before it.
template <typename T>
struct RowView {
  const T* base;      // element e is id e - lead
  int lead, end;
  __device__ RowView(const BeamArgs& p, int row) {
    const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.row_stride;
    lead = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    base = x - lead;
    end = lead + p.vocab;
  }
  // Elements [e0, e0 + N) as fp32, -inf outside the row (which is not read).
  __device__ bool whole(int64_t e0) const { return e0 >= lead && e0 + Vec16<T>::N <= end; }
  __device__ void partial(int64_t e0, float* v) const {
#pragma unroll
    for (int j = 0; j < Vec16<T>::N; ++j) v[j] = e0 + j >= lead && e0 + j < end ? DT<T>::to_f(base[e0 + j]) : -INFINITY;
  }
  __device__ void load(int64_t e0, float* v) const {
    if (whole(e0)) Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4*>(base + e0)), v);
    else partial(e0, v);
  }
};

template <typename T>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamArgs p) {
  constexpr int N = Vec16<T>::N;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  const int64_t row64 = w / p.spans;
  if (row64 >= (int64_t)p.requests * p.beams) return;
  const int row = (int)row64, span = (int)(w - row64 * p.spans);
  if (p.finished && p.finished[row]) return;           // an ended beam: its logits do not count
  const RowView<T> view(p, row);
  const int c0 = span * p.span_chunks, c1 = min(c0 + p.span_chunks, p.chunks);
  if (c0 >= c1) return;
  auto first = [&](int c, int i) { return ((int64_t)c * kChunkVecs + i * 32 + lane) * N; };
  // vectors of the pair of chunks c, c + 1; a lane's raw vector is loaded
  // ahead when it lies whole inside the row
  auto fetch = [&](int c, uint4* raw) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t e0 = first(c, i);
      raw[i] = c + (i >> 1) < c1 && view.whole(e0) ? __ldg(reinterpret_cast<const uint4*>(view.base + e0))
                                                   : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  uint4 raw[4], next[4];
  fetch(c0, raw);
  float m = -INFINITY, sum = 0.f, mine = -INFINITY;
  for (int c = c0; c < c1; c += 2) {
    fetch(c + 2, next);
    float v[4][N], most[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t e0 = first(c, i);
      Vec16<T>::unpack(raw[i], v[i]);
      if (!view.whole(e0) || c + (i >> 1) >= c1) {
        if (c + (i >> 1) < c1) {
          view.partial(e0, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) v[i][j] = -INFINITY;
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) most[i >> 1] = fmaxf(most[i >> 1], v[i][j]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      most[h] = warp_max(most[h]);
      if (lane == c - c0 + h) mine = most[h];
    }
    const float up = fmaxf(most[0], most[1]);
    if (up > m) {                                       // the same in every lane
      sum *= ex2f((m - up) * 1.4426950408889634f);      // 0 the first time
      m = up;
    }
    // a NaN or +inf logit makes the sum NaN: the merge then drops the beam
    const float ref = m == -INFINITY ? 0.f : m;
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) part[i & 1] += ex2f((v[i][j] - ref) * 1.4426950408889634f);
    sum += part[0] + part[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = next[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
  if (lane < c1 - c0) p.maxima[(int64_t)row * p.chunks + c0 + lane] = mine;
  if (lane == 0) p.sums[(int64_t)row * p.spans + span] = make_float2(m, sum);
}

struct MergeSmem {
  double base[kBeamMaxBeams];            // score minus normaliser, -inf: the beam offers nothing
  float basef[kBeamMaxBeams];
  float group[kGroups];
  float bound;
  int chunks, count;
  unsigned long long best;
  uint32_t best_at;
  int chunk[kBeamList];                  // beam * chunks + chunk
  uint64_t value[kBeamList];
  uint32_t at[kBeamList];                // beam * vocab + id
};

// The keep-th largest of the kGroups group maxima (a lower bound of the
// keep-th largest value, -inf if fewer groups have one), less a margin for
// the fp32 values' rounding: a beam's base and its sum with a logit are each
// off by 2^-24 relative, for the element that bounds and the one it is held
// against.
__device__ __forceinline__ void set_bound(MergeSmem& s, float most, int keep, float base_size) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, o));
  if ((tid & 7) == 0) s.group[tid >> 3] = most;
  __syncthreads();
  if (tid < kGroups) {
    const float v = s.group[tid];
    int before = 0;
#pragma unroll 16
    for (int j = 0; j < kGroups; ++j) before += s.group[j] > v || (s.group[j] == v && j < tid);
    if (before == keep - 1) s.bound = v - (fabsf(v) + base_size) * 0x1p-22f;
  }
  __syncthreads();
}

// One CTA per request.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamArgs p) {
  constexpr int N = Vec16<T>::N;
  __shared__ MergeSmem s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x, B = p.beams, K = p.keep;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) s.chunks = s.count = 0;
  __syncthreads();
  // each beam's normaliser: a warp per beam over its spans
  for (int b = warp; b < B; b += kMergeThreads / 32) {
    const int row = r * B + b;
    const double score = (double)p.scores[row];
    double base = score;
    const bool ended = p.finished && p.finished[row];
    if (!ended) {
      const float2* part = p.sums + (int64_t)row * p.spans;
      float m = -INFINITY;
      bool bad = false;
      for (int i = lane; i < p.spans; i += 32) {
        const float2 t = part[i];
        m = fmaxf(m, t.x);
        bad |= !(t.y < INFINITY);
      }
      m = warp_max(m);
      double total = 0.0;
      for (int i = lane; i < p.spans; i += 32) {
        const float2 t = part[i];
        if (t.y > 0.f) total += (double)(t.y * ex2f((t.x - m) * 1.4426950408889634f));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL_MASK, total, o);
      bad = __any_sync(FULL_MASK, bad);
      base = bad || !(total > 0.0) ? -INFINITY : score - ((double)m + log(total));
    }
    const bool finite = base > -INFINITY && base < INFINITY;
    if (lane == 0) {
      s.base[b] = finite ? base : -INFINITY;
      s.basef[b] = finite && !ended ? (float)base : -INFINITY;      // -inf: no logits to look at
      if (finite && ended) {                                         // its one continuation
        const int i = atomicAdd(&s.count, 1);
        s.value[i] = ordered(base + 0.0);
        s.at[i] = (uint32_t)b * p.vocab + p.eos_id;
      }
    }
  }
  __syncthreads();
  const int ended = s.count;
  float base_size = 0.f;
  for (int b = lane; b < B; b += 32) base_size = fmaxf(base_size, s.basef[b] > -INFINITY ? fabsf(s.basef[b]) : 0.f);
  base_size = warp_max(base_size);
  // ---- the chunks that may hold a winner
  const int64_t nc = (int64_t)B * p.chunks;
  auto chunk_value = [&](int64_t c) {
    const int b = (int)(c / p.chunks);
    return s.basef[b] > -INFINITY ? s.basef[b] + p.maxima[(int64_t)r * nc + c] : -INFINITY;
  };
  float most = -INFINITY;
  for (int64_t c = tid; c < nc; c += kMergeThreads) most = fmaxf(most, chunk_value(c));
  set_bound(s, most, K, base_size);
  float bound = s.bound;
  for (int64_t c = tid; c < nc; c += kMergeThreads) {
    const float v = chunk_value(c);
    if (v > -INFINITY && v >= bound) {
      const int i = atomicAdd(&s.chunks, 1);
      if (i < kBeamList) s.chunk[i] = (int)c;
    }
  }
  __syncthreads();
  // calls f(beam, id of the first element, N values) for every vector of those
  // chunks (of all chunks when they are too many to list)
  const bool listed = s.chunks <= kBeamList;
  const int64_t vecs = (listed ? (int64_t)s.chunks : nc) * kChunkVecs;
  auto each = [&](auto f) {
    for (int64_t i = tid; i < vecs; i += kMergeThreads) {
      const int64_t c = listed ? s.chunk[i / kChunkVecs] : i / kChunkVecs;
      const int b = (int)(c / p.chunks);
      if (s.basef[b] == -INFINITY) continue;
      const RowView<T> view(p, r * B + b);
      const int64_t e0 = ((c - (int64_t)b * p.chunks) * kChunkVecs + i % kChunkVecs) * N;
      float v[N];
      view.load(e0, v);
      f(b, (int)e0 - view.lead, v);
    }
  };
  // ---- the bound once more, on their vectors
  most = -INFINITY;
  each([&](int b, int, const float* v) {
    float x = v[0];
#pragma unroll
    for (int j = 1; j < N; ++j) x = fmaxf(x, v[j]);
    most = fmaxf(most, s.basef[b] + x);
  });
  set_bound(s, most, K, base_size);
  bound = fmaxf(bound, s.bound);
  each([&](int b, int id0, const float* v) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float x = s.basef[b] + v[j];
      if (x > -INFINITY && x >= bound) {
        const int i = atomicAdd(&s.count, 1);
        if (i < kBeamList) {
          s.value[i] = ordered(s.base[b] + (double)v[j] + 0.0);
          s.at[i] = (uint32_t)b * p.vocab + (id0 + j);
        }
      }
    }
  });
  __syncthreads();
  auto emit = [&](int k, uint64_t value, uint32_t at) {
    const int64_t o = (int64_t)r * K + k;
    p.out_scores[o] = value ? (float)unordered(value) : -INFINITY;
    p.out_parents[o] = value ? (int)(at / (uint32_t)p.vocab) : -1;
    p.out_tokens[o] = value ? (int)(at % (uint32_t)p.vocab) : -1;
  };
  const int n = s.count;
  if (n <= kBeamList) {
    for (int i = tid; i < n; i += kMergeThreads) {
      const uint64_t value = s.value[i];
      const uint32_t at = s.at[i];
      int before = 0;
      for (int j = 0; j < n; ++j) before += s.value[j] > value || (s.value[j] == value && s.at[j] < at);
      if (before < K) emit(before, value, at);
    }
    for (int i = n + tid; i < K; i += kMergeThreads) emit(i, 0, 0);
    return;
  }
  // so many next to the bound: the best one after the last, keep times
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
    auto offer = [&](uint64_t value, uint32_t at) {
      const bool after = value < last || (value == last && at > last_at);
      if (after && (value > mine || (value == mine && at < mine_at))) mine = value, mine_at = at;
    };
    if (tid < ended) offer(s.value[tid], s.at[tid]);
    each([&](int b, int id0, const float* v) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float x = s.basef[b] + v[j];
        if (x > -INFINITY && x >= bound)
          offer(ordered(s.base[b] + (double)v[j] + 0.0), (uint32_t)b * p.vocab + (id0 + j));
      }
    });
    atomicMax(&s.best, (unsigned long long)mine);
    __syncthreads();
    if (mine && mine == s.best) atomicMin(&s.best_at, mine_at);
    __syncthreads();
    last = s.best;
    last_at = s.best_at;
    if (tid == 0) emit(k, last, last_at);
    __syncthreads();
    if (last == 0) {                                     // nothing left: the rest is empty
      for (int i = k + 1 + tid; i < K; i += kMergeThreads) emit(i, 0, 0);
      break;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const BeamArgs& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.requests * a.beams * a.spans;
  const int64_t ctas = (warps + kScanThreads / 32 - 1) / (kScanThreads / 32);
  cudaError_t e = launch_pdl(beam_scan_kernel<T>, dim3((unsigned)ctas), dim3(kScanThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(beam_merge_kernel<T>, dim3((unsigned)a.requests), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace

// 1 KB chunks of a row, whatever its alignment (a row may start inside its first vector).
int beam_chunks(int dtype, int vocab) {
  const int n = dtype == PKVD_F32 ? 4 : 8;
  const int64_t vecs = ((int64_t)vocab + n - 1 + n - 1) / n;
  return (int)((vecs + kChunkVecs - 1) / kChunkVecs);
}

// A span's sums and a chunk's maximum; at most one span a chunk.
size_t beam_workspace_bytes(int64_t rows, int chunks) {
  return (size_t)rows * chunks * (sizeof(float2) + sizeof(float));
}

cudaError_t launch_beam(const BeamArgs& call, cudaStream_t stream) {
  BeamArgs a = call;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // as many warps as the GPU holds at once (40 an SM), up to 16 chunks each
  const int64_t all = (int64_t)a.requests * a.beams * a.chunks, slots = (int64_t)sms * 40;
  const int64_t each = (all + slots - 1) / slots;
  a.span_chunks = (int)(each < 1 ? 1 : each > kMaxSpan ? kMaxSpan : each);
  a.spans = (a.chunks + a.span_chunks - 1) / a.span_chunks;
  if (a.dtype == PKVD_F32) return launch_typed<float>(a, stream);
  if (a.dtype == PKVD_F16) return launch_typed<__half>(a, stream);
  return launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace pkvd
