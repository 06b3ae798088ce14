// What each cached key was given: the softmax weights of a decode step, summed
// over the query heads of a KV head (or all of them) and added to what earlier
// steps gave.
//   weights_out[i][h][j] = weights[i][h][j] + sum_g 2^(s_gj - M_g) / L_g
//
// A weight needs its row's maximum and sum, which are known when the last key
// has been read.  Reading the keys again would cost half of the attention's
// bytes once more; so the partition kernel leaves the scores it computes anyway
// (4 bytes a query head and key: 1 / 16 of the K/V bytes for 8 query heads a KV
// head of 128 in 16 bits), the merge kernel the rows' statistics, and this kernel,
// bound by bytes, turns scores into weights.  Each element has one thread, so
// no atomics: the sums are the same in every run.
#include "attention_kernels.cuh"

namespace pkvd {

namespace {

constexpr int kThreads = 256, kPer = 4;     // positions of a thread, kThreads apart

// (scores and stats are written by kernels that this one may be scheduled
// beside: plain loads, behind the wait)
__global__ void __launch_bounds__(kThreads) add_weights_kernel(const float* scores, int64_t score_ld,
                                                               const float2* stats, float lift,
                                                               const float* win, float* wout, int64_t seq_stride,
                                                               int64_t head_stride, const int32_t* __restrict__ ctx,
                                                               int ctx_cap, int window, int hq, int group) {
  const int h = blockIdx.y, i = blockIdx.z;
  const int c = min(max(ctx[i], 0), ctx_cap);
  const int base = blockIdx.x * kThreads * kPer + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if ((int)(blockIdx.x * kThreads * kPer) >= c) return;
  const int first = window_start(c, window);
  const float* w = win + (int64_t)i * seq_stride + (int64_t)h * head_stride;
  float* o = wout + (int64_t)i * seq_stride + (int64_t)h * head_stride;
  float sum[kPer], before[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int j = base + k * kThreads;
    sum[k] = 0.f;
    before[k] = j < c ? w[j] : 0.f;
  }
  const int64_t row0 = (int64_t)i * hq + (int64_t)h * group;
#pragma unroll 8
  for (int g = 0; g < group; ++g) {
    const float2 st = stats[row0 + g];
    const float* s = scores + (row0 + g) * score_ld;
    const float m = st.x - lift;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = base + k * kThreads;
      if (j >= first && j < c) sum[k] = fmaf(exp2f(s[j] - m), st.y, sum[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int j = base + k * kThreads;
    if (j < c) o[j] = before[k] + sum[k];
  }
}

}  // namespace

int64_t score_row(int max_context_len) { return ((int64_t)max_context_len + 7) / 8 * 8; }

cudaError_t launch_attention_weights(const AttnArgs& a, const WeightArgs& w, cudaStream_t stream) {
  cudaError_t e = launch_attention(a, stream);
  if (e != cudaSuccess || a.grid == 0) return e;
  const long long cap = (long long)a.max_blocks_per_seq * a.block_size;
  const int ctx_cap = (int)(cap < a.max_context_len ? cap : a.max_context_len);
  // f16 weights are lifted in the partition kernel's sums on the tensor cores
  const float lift = a.path == PKVD_PATH_MMA && a.dtype == PKVD_F16 ? kWeightLift<__half> : 0.f;
  const int span = kThreads * kPer;
  const dim3 grid((unsigned)((ctx_cap + span - 1) / span), (unsigned)w.heads, (unsigned)a.num_seqs);
  return launch_pdl(add_weights_kernel, grid, dim3(kThreads), 0, stream, (const float*)a.scores, a.score_ld,
                    (const float2*)a.stats, lift, w.in, w.out, w.seq_stride, w.head_stride, a.context_lens, ctx_cap,
                    a.window, a.num_q_heads, a.num_q_heads / w.heads);
}

}  // namespace pkvd
