// Internal launchers shared between the kernel translation units and the
// C-ABI layer (api.cu).  Host-side argument validation happens in api.cu;
// these functions only size grids and enqueue kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pkvd.h"

namespace pkvd {

// Decode-attention launch geometry shared by the workspace query and the
// launcher, so both derive the same grid.
constexpr int kChunk = 16;            // tokens per pipeline stage
constexpr int kConsumerWarps = 8;
constexpr int kAttnThreads = (kConsumerWarps + 1) * 32;

// Scores capped by a tanh, biased by distance or opened to a prefix
// (score_mod.cuh); all off by default.
struct ScoreMod {
  float cap_in = 0.f;            // softmax scale / cap, 0: no cap
  float cap_out_log2 = 0.f;      // cap * log2(e)
  const float* slopes = nullptr;     // [query heads]
  const int32_t* prefix = nullptr;   // [sequences], prefill only
  bool on() const { return cap_in != 0.f || slopes || prefix; }
};

struct AttnArgs {
  void* out;
  const void* q;
  const void* k_base;
  const void* v_base;
  int64_t block_stride, token_stride, head_stride;  // elements
  int64_t num_blocks;
  int block_size;
  int num_kv_heads;
  int num_q_heads;
  int head_dim;
  int dtype;
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* context_lens;
  int max_context_len;
  int num_seqs;
  float scale;
  void* workspace;
  int32_t* err;
  int grid;           // partition CTAs
  int path;           // PKVD_PATH_FMA / PKVD_PATH_MMA (resolved)
  int window;         // > 0: sliding window of the newest `window` positions
  ScoreMod mod;
  // Set where every key's score is handed on (launch_attention_weights): scores
  // [num_seqs][num_q_heads][score_ld], pairs (maximum, 1 / sum) [num_seqs][num_q_heads]
  float* scores = nullptr;
  int64_t score_ld = 0;
  float* stats = nullptr;
};

// Decode attention that also counts what each key was given (attention_weights.cu).
struct WeightArgs {
  const float* in;         // [num_seqs][heads][length], rows at these strides
  float* out;
  int64_t seq_stride, head_stride;
  int heads;               // 1 or the KV heads
};
int64_t score_row(int max_context_len);      // scores of one head's row in the workspace
cudaError_t launch_attention_weights(const AttnArgs& a, const WeightArgs& w, cudaStream_t stream);

// Rows of the cache close up (compact.cu).
struct CompactArgs {
  void* k_base;
  void* v_base;
  int64_t block_stride, token_stride, head_stride, num_blocks;   // elements
  int block_size, block_shift, num_kv_heads, head_dim, elem_bytes;
  const int32_t* tables;
  const int32_t* new_tables;    // the same pointer: in place
  int max_blocks, new_max_blocks;
  int max_tokens, new_max_tokens;
  const int32_t* positions;     // strides in elements; head stride 0: alike for all heads
  int64_t pos_stride, pos_head_stride;
  const int32_t* counts;
  const int32_t* first;         // or null: 0
  int max_count;
  int32_t* err;
};
cudaError_t launch_compact(const CompactArgs& a, int num_seqs, cudaStream_t stream);

// Which positions stay (evict.cu).
struct EvictArgs {
  const float* weights;         // [num_seqs][heads][length]
  float* weights_out;           // or null
  int64_t seq_stride, head_stride;
  int length;
  const int32_t* context_lens;
  int keep, sink, recent;
  int32_t* positions;           // [num_seqs][heads][keep]
  int32_t* counts;              // [num_seqs]
  int32_t* err;
};
cudaError_t launch_evict_select(const EvictArgs& a, int num_seqs, int heads, cudaStream_t stream);

// Attention of drafted trees (tree.cu, tree_tc.cu).
constexpr int kTreeMaxNodes = 256;    // nodes of a sequence's tree
constexpr int kTreeKeys = 128;        // keys of a tile
constexpr int kTreeFewRows = 64;      // (node, query head) rows of a tree that tree_few.cu takes
struct TreeArgs {
  void* out;
  const void* q;
  pkvd_cache cache;
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  const int32_t* parents;
  int num_seqs, total_q, max_seqlen_q, num_q_heads;
  float scale;
  int window;
  ScoreMod mod;
  void* workspace;
  int32_t* err;
  int path;                // PKVD_PATH_FMA / PKVD_PATH_TC (resolved)
  int sms;
};
bool tree_tc_supported(const TreeArgs& a);
size_t tree_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int max_seqlen_q, int sms);
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream);

// Which drafted nodes the target's choices follow (tree.cu).
struct AcceptArgs {
  const int32_t* drafted;
  const int32_t* parents;
  const int32_t* target;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int total_q, max_path;
  int32_t* positions;      // [num_seqs][max_path]
  int32_t* first;
  int32_t* counts;
  int32_t* tokens;         // [num_seqs][max_path]
  int32_t* err;
};
cudaError_t launch_tree_accept(const AcceptArgs& a, int num_seqs, cudaStream_t stream);

int attention_grid(int num_seqs, int max_context_len, int sm_count);
size_t attention_workspace_bytes(int num_seqs, int num_q_heads, int head_dim, int grid);
bool attention_path_supported(int path, int dtype, int head_dim, int num_kv_heads, int group);
int attention_default_path(int dtype, int head_dim, int num_kv_heads, int group);
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream);
// Rows sharing their first prefix_len cached tokens (attention_prefix.cu):
// whether the shared-prefix kernel takes such a call, its workspace, and the
// launch (partition + merge).
bool prefix_path_usable(int dtype, int head_dim, int num_kv_heads, int num_q_heads, int num_seqs, int grid,
                        int prefix_len, int window);
size_t prefix_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int grid,
                              int prefix_len);
cudaError_t launch_attention_prefix(const AttnArgs& a, int prefix_len, cudaStream_t stream);
// Host-side checks of a decode attention call (api.cu), shared by every
// attention entry point: resolves PKVD_PATH_AUTO in *path and, for a call
// with rows, gives the partition grid and the workspace bytes it needs.
// Checks nothing about the workspace itself.
pkvd_status attention_validate(void* out, const void* q, const pkvd_cache* cache, const int32_t* block_tables,
                               int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t max_context_len,
                               int32_t num_seqs, int32_t num_q_heads, float scale, int32_t window, int32_t* path,
                               int* grid, size_t* need);

cudaError_t launch_slot_mapping(int64_t* slots, const int32_t* tables, int max_blocks,
                                const int32_t* ctx, int num_seqs, int block_size,
                                int64_t num_blocks, cudaStream_t stream, int32_t* err);

cudaError_t launch_kv_store(const void* k, const void* v, const int64_t* slots, int num_tokens,
                            const pkvd_cache& c, int elem_bytes, cudaStream_t stream,
                            int32_t* err);
cudaError_t launch_kv_store_paged(const void* k, const void* v, const int32_t* tables, int max_blocks,
                                  const int32_t* ctx, int num_seqs, int64_t* slots_out, const pkvd_cache& c,
                                  int elem_bytes, cudaStream_t stream, int32_t* err);
cudaError_t launch_copy_blocks(const pkvd_cache& c, int elem_bytes, const int32_t* src, const int32_t* dst,
                               const int32_t* rows, int count, cudaStream_t stream, int32_t* err);

// Varlen paged prefill (prefill.cu, store.cu).
struct PrefillArgs {
  void* out;
  const void* q;
  pkvd_cache cache;
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  int num_seqs;
  int total_q;
  int max_seqlen_q;
  int num_q_heads;
  float scale;
  int window;
  ScoreMod mod;
  int32_t* err;
};
bool prefill_supported(int dtype, int head_dim, int group);
bool prefill_tc_supported(const PrefillArgs& a);
bool prefill_fma_supported(int dtype, int head_dim, int group, int num_kv_heads);
cudaError_t launch_prefill_fma(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_tc(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_mod(const PrefillArgs& a, cudaStream_t stream);   // with score modifiers
int prefill_tile_tokens(int group);
cudaError_t launch_prefill_attention(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_kv_store_prefill(const void* k, const void* v, const int32_t* tables, int max_blocks,
                                    const int32_t* cu_q, const int32_t* cu_k, int num_seqs, int total_q,
                                    int64_t* slots_out, const pkvd_cache& c, int elem_bytes, cudaStream_t stream,
                                    int32_t* err);

// Rotary positions, alone (positions set) or with the paged store of a decode
// step (ctx set) or of a prefill batch (cu_q and cu_k set): rope.cu.  Strides
// in elements; k_out and v_out are the cache bases in the store forms.
constexpr int kRopeMaxDim = 512;      // largest head_dim
struct RopeArgs {
  void* q_out;
  const void* q;
  void* k_out;
  const void* k;
  void* v_out;
  const void* v;
  int64_t q_stride, q_out_stride, k_stride, k_out_stride, v_stride;
  int64_t block_stride, token_stride, head_stride, num_blocks;
  int block_size;
  int dtype;
  int num_q_heads, num_kv_heads, head_dim;
  int rotary_dim, interleaved;
  float mscale;
  const double* inv_freq;
  const int64_t* positions;
  const int32_t* tables;
  int max_blocks;
  const int32_t* ctx;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int num_seqs;
  int64_t* slots_out;
  int32_t* err;
  int num_tokens, parts, part_heads;   // set by launch_rope: warps of a token, heads of a warp
};
cudaError_t launch_rope(const RopeArgs& a, int tokens, cudaStream_t stream);

// One step of beam search (beam.cu).
constexpr int kBeamMaxKeep = 64;      // continuations kept per request
constexpr int kBeamMaxBeams = 64;     // beams per request
struct BeamArgs {
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  const void* logits;
  int dtype;
  int requests, beams, vocab, keep;
  int64_t row_stride;
  const float* scores;
  const uint8_t* finished;
  int eos_id;
  int chunks;           // 1 KB chunks of a row
  int span_chunks, spans;   // chunks a warp scans, spans of a row (set by launch_beam)
  uint32_t chunk_mul;   // n / chunks = (umulhi(n, chunk_mul) + n) >> chunk_shift
  int chunk_shift;
  float4* sums;         // workspace: [rows][spans] maximum, sum of exponentials (two parts)
  float* maxima;        // then (behind [rows][chunks] of the former) [rows][chunks]
};
int beam_chunks(int dtype, int vocab);
size_t beam_workspace_bytes(int64_t rows, int chunks);
cudaError_t launch_beam(const BeamArgs& a, cudaStream_t stream);

// Per-row cut parameters the sampler leaves for the extras kernel:
// [0] flags (kRowGreedy, kRowUniform, kRowTopK), [1] nucleus threshold key
// (0 = off), [2] k-th key, [3] index of the last kept id at the k-th key
// (INT_MAX: every one), [4] the row max value (f32 bits), [5..7] unused.
constexpr int kRowInfo = 8;
constexpr int kRowGreedy = 1, kRowUniform = 2, kRowTopK = 4;

// One sampler call's arguments, for the two builds of the sampler kernel
// (sampler.cu: 1024-thread CTAs; sampler512.cu: 512-thread CTAs).
struct SampleCall {
  int32_t* token_ids;
  const void* logits;
  int dtype;
  int num_rows;
  int vocab;
  int64_t row_stride;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const uint64_t* seeds;
  const uint64_t* offsets;
  const uint32_t* mask;
  int64_t mask_stride;
  int32_t* row_info;
};
// Each build: launch (or, with waves_only, only report how many waves of
// clusters it would need), and whether a masked row fits on chip.
namespace s1024 {
cudaError_t sample_launch(const SampleCall& c, cudaStream_t stream, int* waves_only);
bool sample_mask_fits(int dtype, int vocab, int64_t row_stride, const void* logits);
}  // namespace s1024
namespace s512 {
cudaError_t sample_launch(const SampleCall& c, cudaStream_t stream, int* waves_only);
bool sample_mask_fits(int dtype, int vocab, int64_t row_stride, const void* logits);
}  // namespace s512

cudaError_t launch_sample(int32_t* token_ids, const void* logits, int dtype, int num_rows,
                          int vocab, int64_t row_stride, const float* temperature,
                          const int32_t* top_k, const float* top_p, const uint64_t* seeds,
                          const uint64_t* offsets, const uint32_t* mask, int64_t mask_stride,
                          int32_t* row_info, cudaStream_t stream);
bool sample_mask_supported(int dtype, int vocab, int64_t row_stride, const void* logits);
cudaError_t launch_sample_extras(const void* logits, int dtype, int num_rows, int vocab, int64_t row_stride,
                                 const float* temperature, const uint32_t* mask, int64_t mask_stride,
                                 const int32_t* row_info, const int32_t* token_ids, float* token_prob,
                                 float* top_probs, int32_t* top_ids, cudaStream_t stream);

int device_sm_count();   // current device, cached; <= 0 on failure
int64_t device_l2_bytes();   // current device's L2 size in bytes, cached; 0 on failure

}  // namespace pkvd
