// Host-side launchers of the PBD kernels (internal to the library; the public C ABI is
// include/la_pbd.h).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "la_pbd.h"
#include "pbd_common.cuh"

namespace la {

// Launch with programmatic stream serialization allowed (see pdl_wait in pbd_common.cuh).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                             const int32_t* seq_lens, const int32_t* window_lens, int B, int W,
                             int Hkv, int S, cudaStream_t stream);

// Empty kernel with programmatic dependent launch (launch-floor measurements).
cudaError_t launch_noop(int ctas, int threads, cudaStream_t stream);

// CUDA-core split-KV attention (any R = W * G <= 128).
int simt_rows_per_thread(int R);
int simt_tile_keys();
size_t simt_smem_bytes(int R, int B);
cudaError_t simt_max_ctas_per_sm(int R, int B, int* ctas);
cudaError_t launch_attn_simt(const Problem& p, cudaStream_t stream);

// tcgen05 + TMA split-KV attention (R <= 80).
size_t tc_smem_bytes(int R, int B);
cudaError_t launch_attn_tc(const Problem& p, const void* tmap_k, const void* tmap_v,
                           const void* tmap_q, const void* tmap_o, cudaStream_t stream);

// tcgen05 + TMA block-causal prefill (one CTA per 128 query rows of a (sequence, head)).
size_t prefill_smem_bytes();
// Launches the V conversion (prefill_v16_kernel) and then the prefill kernel.
cudaError_t launch_prefill_tc(const PrefillProblem& p, const void* tmap_q, const void* tmap_k,
                              const void* tmap_v, const void* tmap_v16, cudaStream_t stream);

// Merge of the per-split partials into the bf16 output.
cudaError_t launch_combine(const Problem& p, cudaStream_t stream);

// Host-side checks and choices shared by the C ABI's files (la_pbd_api.cu).
la_status check_cfg(const la_pbd_cfg* cfg, int32_t window_len);
cudaError_t sm_count(int* out);

// Attention weights of the keys (second half of la_pbd_attn_weights): see key_weights.cu.
struct KeyWeights {
  const float* lse2;            // [B * Hkv, rows_pad], from the attention and merge kernels
  const float* in;              // [B, Hkv, S] or null (zeros)
  float* out;                   // [B, Hkv, S]; may be `in`
  float decay;
};
cudaError_t launch_key_weights(const Problem& p, const KeyWeights& kw, const void* tmap_k,
                               const void* tmap_q, cudaStream_t stream);

// Rotation alone: x, out [tokens, heads, head_dim] with strides in elements.
struct RopeProblem {
  const void* x;
  void* out;
  const int32_t* positions;     // [tokens]
  long long tokens, x_tok, x_head, y_tok, y_head;
  int heads, head_dim;
  bool inverse;
};
cudaError_t launch_rope(const la_rope_plan& plan, const RopeProblem& p, int dtype, int sms,
                        cudaStream_t stream);

// Rotation and append of T rows a sequence.
struct RopeAppendProblem {
  const __nv_bfloat16 *q, *k_new, *v_new;   // [B, T, heads, D], a token's stride in elements
  long long q_tok, k_tok, v_tok;
  const int32_t *seq_lens, *row_lens, *pos0;   // [B], each may be null
  __nv_bfloat16 *q_out, *kc, *vc;
  int32_t* key_pos;             // [B, Hkv, S] or null
  const int32_t* block_table;   // null: contiguous caches
  int pages_per_seq, page_size, num_pages;
  int B, T, Hq, Hkv, S;         // S = key slots of a sequence
};
cudaError_t launch_rope_append(const la_rope_plan& plan, const RopeAppendProblem& p, int sms,
                               cudaStream_t stream);

// Eviction: see kv_evict.cu.
constexpr int kMaxEvictCtas = 8;
struct EvictList {              // of a (sequence, KV head): where each CTA's holes and movers end
  int holes[kMaxEvictCtas], movers[kMaxEvictCtas];
};
struct EvictProblem {
  const float* weights;         // [B, Hkv, S]
  const int32_t *key_pos, *seq_lens, *next_pos;   // [B, Hkv, S] or null, [B], [B] or null
  __nv_bfloat16 *kc, *vc;
  const int32_t* block_table;
  int pages_per_seq, page_size, num_pages;
  float* weights_out;
  int32_t *key_pos_out, *kept_slots, *new_lens;   // the first two may be null
  WsHeader* hdr;
  EvictList* lists;             // [B * Hkv]
  int *moves, *kept_lens, *lens;   // [B * Hkv] keys that change place, keys that stay; [B] new lengths
  uint32_t* hole_bits;          // [B * Hkv, bit_words]: evicted slots, a bit each
  int bit_words;                // of a head: slots of all CTAs' parts / 32
  int* slots;                   // [B * Hkv, CTAs, 2, part]: holes, movers
  int B, Hkv, S, budget, sink, recent;
  int part;                     // most keys of a CTA
};
int evict_ctas(int S, int heads);   // CTAs of a (sequence, KV head)
int evict_part(int S, int heads);
cudaError_t launch_evict(const EvictProblem& p, int sms, cudaStream_t stream);

// Verification of drafted tokens: see verify.cu. Strides in elements.
struct VerifyProblem {
  const void *p, *q;            // rows of V; q may be null
  long long p_batch, p_row, q_batch, q_row;
  const int32_t *drafts, *draft_lens, *seq_lens;
  const float *u, *sample_u;
  int32_t *tokens, *accepted, *seq_lens_out;
  int B, K, V;
};
cudaError_t launch_verify(const VerifyProblem& p, int dtype, int sms, cudaStream_t stream);

// Workspace carve-up shared by the launchers and the C ABI.
constexpr size_t kPrefixOffset = kHeaderBytes;                               // int[B+1]
constexpr size_t kPrefixBytes = ((size_t)(kMaxBatch + 1) * 4 + 255) / 256 * 256;
constexpr size_t kSlotsOffset = kPrefixOffset + kPrefixBytes;
constexpr int kMaxCtasPerSm = 4;

}  // namespace la
