// C ABI of the operators around the window attention (declared in include/la_pbd.h): rotary
// positions, eviction and draft verification. Argument validation, workspace carve-up and launch;
// nothing here allocates device memory or synchronises.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "la_pbd.h"
#include "pbd_common.cuh"
#include "pbd_kernels.h"

namespace {

using la::check_cfg;

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kMaxRotary = 256;
constexpr int kMaxDrafts = 32;

la_status check_plan(const la_rope_plan* pl, int head_dim) {
  if (!pl) return LA_ERR_INVALID_ARG;
  if (pl->layout != LA_ROPE_HALF && pl->layout != LA_ROPE_INTERLEAVED) return LA_ERR_INVALID_ARG;
  if (pl->rotary_dim < 2 || pl->rotary_dim > kMaxRotary || pl->rotary_dim % 2 != 0 ||
      pl->rotary_dim > head_dim)
    return LA_ERR_INVALID_ARG;
  return LA_OK;
}

// Page pool arguments, as for the paged attention.
la_status check_pages(const la_pbd_cfg* cfg, const int32_t* block_table, int32_t pages_per_seq,
                      int32_t page_size, int32_t num_pages) {
  if (!block_table || !aligned(block_table, 4)) return LA_ERR_INVALID_ARG;
  if (pages_per_seq < 1 || num_pages < 1 || page_size < 64 || page_size % 64 != 0)
    return LA_ERR_INVALID_ARG;
  if ((long long)num_pages * cfg->num_kv_heads * page_size >= (1LL << 31)) return LA_ERR_UNSUPPORTED;
  if ((long long)cfg->batch * cfg->num_kv_heads * pages_per_seq * page_size >= (1LL << 31))
    return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

}  // namespace

extern "C" {

la_status la_rope_plan_init(la_rope_plan* plan, int32_t rotary_dim, int32_t layout, int32_t scaling,
                            double base, double factor, int32_t original_max, double low_turns,
                            double high_turns, float out_scale) {
  if (!plan) return LA_ERR_INVALID_ARG;
  if (layout != LA_ROPE_HALF && layout != LA_ROPE_INTERLEAVED) return LA_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim > kMaxRotary || rotary_dim % 2 != 0) return LA_ERR_INVALID_ARG;
  if (scaling < LA_ROPE_SCALE_NONE || scaling > LA_ROPE_SCALE_TURNS) return LA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(out_scale)) return LA_ERR_INVALID_ARG;
  if (scaling != LA_ROPE_SCALE_NONE && (!std::isfinite(factor) || factor <= 0.0)) return LA_ERR_INVALID_ARG;
  const bool ramp = scaling == LA_ROPE_SCALE_PAIRS || scaling == LA_ROPE_SCALE_TURNS;
  if (ramp && (original_max < 1 || !std::isfinite(low_turns) || !std::isfinite(high_turns) ||
               low_turns <= 0.0 || high_turns <= low_turns))
    return LA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const int pairs = rotary_dim / 2;
  if (scaling == LA_ROPE_SCALE_BASE && rotary_dim > 2)
    base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
  if (!std::isfinite(base) || base <= 0.0) return LA_ERR_INVALID_ARG;
  // The pairs that turn high_turns and low_turns times over the original length.
  double lo = 0.0, hi = 1.0;
  if (scaling == LA_ROPE_SCALE_PAIRS) {
    auto pair_of = [&](double turns) {
      return rotary_dim * std::log(original_max / (turns * two_pi)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(high_turns)), 0.0);
    hi = std::fmin(std::ceil(pair_of(low_turns)), (double)(rotary_dim - 1));
  }
  std::memset(plan, 0, sizeof(*plan));
  plan->rotary_dim = rotary_dim;
  plan->layout = layout;
  plan->out_scale = out_scale;
  for (int i = 0; i < pairs; ++i) {
    double w = std::pow(base, -2.0 * i / rotary_dim);   // angle per position
    double keep = 1.0;                                  // share that is not scaled
    if (scaling == LA_ROPE_SCALE_LINEAR) keep = 0.0;
    if (scaling == LA_ROPE_SCALE_PAIRS)
      keep = 1.0 - std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
    if (scaling == LA_ROPE_SCALE_TURNS) {
      const double turns = original_max * w / two_pi;
      keep = std::fmin(std::fmax((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0);
    }
    if (keep < 1.0) w = keep * w + (1.0 - keep) * w / factor;
    plan->turns[i] = w / two_pi;
  }
  return LA_OK;
}

la_status la_rope(const la_rope_plan* plan, int32_t dtype, const void* x, int64_t x_token_stride,
                  int64_t x_head_stride, const int32_t* positions, int64_t tokens, int32_t heads,
                  int32_t head_dim, int32_t inverse, void* out, int64_t out_token_stride,
                  int64_t out_head_stride, void* stream) {
  if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_F16) return LA_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 1 || head_dim < 2) return LA_ERR_INVALID_ARG;
  if (head_dim % 2 != 0 || head_dim > kMaxRotary) return LA_ERR_UNSUPPORTED;
  la_status st = check_plan(plan, head_dim);
  if (st != LA_OK) return st;
  if (tokens >= (1LL << 31) || (long long)heads * head_dim >= (1LL << 20)) return LA_ERR_UNSUPPORTED;
  if (tokens == 0) return LA_OK;
  const uintptr_t es = dtype == LA_DTYPE_F32 ? 4 : 2;
  if (!x || !out || !positions || !aligned(x, es) || !aligned(out, es) || !aligned(positions, 4))
    return LA_ERR_INVALID_ARG;
  // Rows of the output must not overlap: tokens outside heads or the other way round.
  if (x_token_stride < 0 || x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0)
    return LA_ERR_INVALID_ARG;
  if (heads > 1 && out_head_stride < head_dim) return LA_ERR_INVALID_ARG;
  if (tokens > 1) {
    const long long of_token = (heads - 1LL) * out_head_stride + head_dim;
    const long long of_head = (tokens - 1LL) * out_token_stride + head_dim;
    if (out_token_stride < head_dim ||
        (heads > 1 && out_token_stride < of_token && out_head_stride < of_head))
      return LA_ERR_INVALID_ARG;
  }
  if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return LA_ERR_INVALID_ARG;
  la::RopeProblem p;
  p.x = x;
  p.out = out;
  p.positions = positions;
  p.tokens = tokens;
  p.x_tok = x_token_stride;
  p.x_head = x_head_stride;
  p.y_tok = out_token_stride;
  p.y_head = out_head_stride;
  p.heads = heads;
  p.head_dim = head_dim;
  p.inverse = inverse != 0;
  int sms = 0;
  if (la::sm_count(&sms) != cudaSuccess) return LA_ERR_CUDA;
  return la::launch_rope(*plan, p, dtype, sms, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"

namespace {

struct Pages {
  const int32_t* block_table = nullptr;
  int32_t pages_per_seq = 0, page_size = 0, num_pages = 0;
};

la_status rope_append(const la_pbd_cfg* cfg, const la_rope_plan* plan, const void* q, int64_t q_tok,
                      const void* k_new, int64_t k_tok, const void* v_new, int64_t v_tok,
                      const int32_t* seq_lens, const int32_t* row_lens, const int32_t* pos0,
                      int32_t rows, void* q_out, void* kc, void* vc, int32_t* key_pos, const Pages& pg,
                      void* stream) {
  la_status st = check_plan(plan, la::kHeadDim);
  if (st != LA_OK) return st;
  if (rows < 1) return LA_ERR_INVALID_ARG;
  if ((long long)cfg->batch * rows >= (1LL << 30)) return LA_ERR_UNSUPPORTED;
  if (!q || !k_new || !v_new || !q_out || !kc || !vc) return LA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16) ||
      !aligned(kc, 16) || !aligned(vc, 16) || !aligned(seq_lens, 4) || !aligned(row_lens, 4) ||
      !aligned(pos0, 4) || !aligned(key_pos, 4))
    return LA_ERR_INVALID_ARG;
  const int64_t dq = (int64_t)cfg->num_q_heads * la::kHeadDim, dk = (int64_t)cfg->num_kv_heads * la::kHeadDim;
  if (q_tok < dq || k_tok < dk || v_tok < dk || q_tok % 8 || k_tok % 8 || v_tok % 8)
    return LA_ERR_INVALID_ARG;
  // In place only with the same layout: q_out is dense.
  if (q == q_out && q_tok != dq) return LA_ERR_INVALID_ARG;
  la::RopeAppendProblem p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.q_tok = q_tok;
  p.k_tok = k_tok;
  p.v_tok = v_tok;
  p.seq_lens = seq_lens;
  p.row_lens = row_lens;
  p.pos0 = pos0;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.kc = static_cast<__nv_bfloat16*>(kc);
  p.vc = static_cast<__nv_bfloat16*>(vc);
  p.key_pos = key_pos;
  p.block_table = pg.block_table;
  p.pages_per_seq = pg.pages_per_seq;
  p.page_size = pg.page_size;
  p.num_pages = pg.num_pages;
  p.B = cfg->batch;
  p.T = rows;
  p.Hq = cfg->num_q_heads;
  p.Hkv = cfg->num_kv_heads;
  p.S = pg.block_table ? pg.pages_per_seq * pg.page_size : cfg->max_seq;
  int sms = 0;
  if (la::sm_count(&sms) != cudaSuccess) return LA_ERR_CUDA;
  return la::launch_rope_append(*plan, p, sms, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

// Workspace of la_kv_evict: header, lists' ends, moves, lengths, hole bits, lists.
struct EvictWs {
  size_t lists, moves, kept_lens, lens, bits, slots, total;
  int ctas, part, bit_words;
};
EvictWs evict_ws(const la_pbd_cfg* cfg, int S) {
  const size_t heads = (size_t)cfg->batch * cfg->num_kv_heads;
  EvictWs w;
  w.ctas = la::evict_ctas(S, (int)heads);
  w.part = la::evict_part(S, (int)heads);
  w.bit_words = w.ctas * w.part / 32;
  w.lists = la::kHeaderBytes;
  w.moves = w.lists + heads * sizeof(la::EvictList);
  w.kept_lens = w.moves + heads * sizeof(int);
  w.lens = w.kept_lens + heads * sizeof(int);
  w.bits = w.lens + (size_t)cfg->batch * sizeof(int);
  w.slots = w.bits + heads * w.bit_words * sizeof(uint32_t);
  w.total = w.slots + heads * w.ctas * 2 * (size_t)w.part * sizeof(int);
  // Every workspace is at least what la_pbd_workspace_init takes.
  if (w.total < la::kSlotsOffset) w.total = la::kSlotsOffset;
  return w;
}

la_status kv_evict(const la_pbd_cfg* cfg, const float* weights, const int32_t* key_pos,
                   const int32_t* seq_lens, const int32_t* next_pos, int32_t budget, int32_t sink,
                   int32_t recent, void* kc, void* vc, float* weights_out, int32_t* key_pos_out,
                   int32_t* kept_slots, int32_t* new_lens, const Pages& pg, void* workspace,
                   size_t workspace_bytes, void* stream) {
  const int S = pg.block_table ? pg.pages_per_seq * pg.page_size : cfg->max_seq;
  if (budget < 1 || budget > S || sink < 0 || recent < 0 || (long long)sink + recent > budget)
    return LA_ERR_INVALID_ARG;
  if (!weights || !seq_lens || !kc || !vc || !weights_out || !new_lens) return LA_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(key_pos, 4) || !aligned(seq_lens, 4) || !aligned(next_pos, 4) ||
      !aligned(kc, 16) || !aligned(vc, 16) || !aligned(weights_out, 4) || !aligned(key_pos_out, 4) ||
      !aligned(kept_slots, 4) || !aligned(new_lens, 4))
    return LA_ERR_INVALID_ARG;
  // Positions that are kept must be kept up to date.
  if (key_pos && !key_pos_out) return LA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return LA_ERR_WORKSPACE;
  const EvictWs w = evict_ws(cfg, S);
  if (workspace_bytes < w.total) return LA_ERR_WORKSPACE;
  int sms = 0;
  if (la::sm_count(&sms) != cudaSuccess) return LA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  la::EvictProblem p;
  std::memset(&p, 0, sizeof(p));
  p.weights = weights;
  p.key_pos = key_pos;
  p.seq_lens = seq_lens;
  p.next_pos = next_pos;
  p.kc = static_cast<__nv_bfloat16*>(kc);
  p.vc = static_cast<__nv_bfloat16*>(vc);
  p.block_table = pg.block_table;
  p.pages_per_seq = pg.pages_per_seq;
  p.page_size = pg.page_size;
  p.num_pages = pg.num_pages;
  p.weights_out = weights_out;
  p.key_pos_out = key_pos_out;
  p.kept_slots = kept_slots;
  p.new_lens = new_lens;
  p.hdr = reinterpret_cast<la::WsHeader*>(ws);
  p.lists = reinterpret_cast<la::EvictList*>(ws + w.lists);
  p.moves = reinterpret_cast<int*>(ws + w.moves);
  p.kept_lens = reinterpret_cast<int*>(ws + w.kept_lens);
  p.lens = reinterpret_cast<int*>(ws + w.lens);
  p.hole_bits = reinterpret_cast<uint32_t*>(ws + w.bits);
  p.bit_words = w.bit_words;
  p.slots = reinterpret_cast<int*>(ws + w.slots);
  p.B = cfg->batch;
  p.Hkv = cfg->num_kv_heads;
  p.S = S;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.part = w.part;
  return la::launch_evict(p, sms, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // namespace

extern "C" {

la_status la_rope_append(const la_pbd_cfg* cfg, const la_rope_plan* plan, const void* q,
                         int64_t q_token_stride, const void* k_new, int64_t k_token_stride,
                         const void* v_new, int64_t v_token_stride, const int32_t* seq_lens,
                         const int32_t* row_lens, const int32_t* pos0, int32_t rows, void* q_out,
                         void* k_cache, void* v_cache, int32_t* key_pos, void* stream) {
  la_status st = check_cfg(cfg, 1);
  if (st != LA_OK) return st;
  return rope_append(cfg, plan, q, q_token_stride, k_new, k_token_stride, v_new, v_token_stride, seq_lens,
                     row_lens, pos0, rows, q_out, k_cache, v_cache, key_pos, Pages(), stream);
}

la_status la_rope_append_paged(const la_pbd_cfg* cfg, const la_rope_plan* plan, const void* q,
                               int64_t q_token_stride, const void* k_new, int64_t k_token_stride,
                               const void* v_new, int64_t v_token_stride, const int32_t* block_table,
                               int32_t pages_per_seq, int32_t page_size, int32_t num_pages,
                               const int32_t* seq_lens, const int32_t* row_lens, const int32_t* pos0,
                               int32_t rows, void* q_out, void* k_pool, void* v_pool, int32_t* key_pos,
                               void* stream) {
  la_status st = check_cfg(cfg, 1);
  if (st == LA_OK) st = check_pages(cfg, block_table, pages_per_seq, page_size, num_pages);
  if (st != LA_OK) return st;
  Pages pg{block_table, pages_per_seq, page_size, num_pages};
  return rope_append(cfg, plan, q, q_token_stride, k_new, k_token_stride, v_new, v_token_stride, seq_lens,
                     row_lens, pos0, rows, q_out, k_pool, v_pool, key_pos, pg, stream);
}

size_t la_kv_evict_workspace_bytes(const la_pbd_cfg* cfg) {
  if (check_cfg(cfg, 1) != LA_OK) return 0;
  return evict_ws(cfg, cfg->max_seq).total;
}

la_status la_kv_evict(const la_pbd_cfg* cfg, const float* weights, const int32_t* key_pos,
                      const int32_t* seq_lens, const int32_t* next_pos, int32_t budget, int32_t sink,
                      int32_t recent, void* k_cache, void* v_cache, float* weights_out,
                      int32_t* key_pos_out, int32_t* kept_slots, int32_t* new_lens, void* workspace,
                      size_t workspace_bytes, void* stream) {
  la_status st = check_cfg(cfg, 1);
  if (st != LA_OK) return st;
  return kv_evict(cfg, weights, key_pos, seq_lens, next_pos, budget, sink, recent, k_cache, v_cache,
                  weights_out, key_pos_out, kept_slots, new_lens, Pages(), workspace, workspace_bytes, stream);
}

la_status la_kv_evict_paged(const la_pbd_cfg* cfg, const float* weights, const int32_t* key_pos,
                            const int32_t* block_table, int32_t pages_per_seq, int32_t page_size,
                            int32_t num_pages, const int32_t* seq_lens, const int32_t* next_pos,
                            int32_t budget, int32_t sink, int32_t recent, void* k_pool, void* v_pool,
                            float* weights_out, int32_t* key_pos_out, int32_t* kept_slots,
                            int32_t* new_lens, void* workspace, size_t workspace_bytes, void* stream) {
  la_status st = check_cfg(cfg, 1);
  if (st == LA_OK) st = check_pages(cfg, block_table, pages_per_seq, page_size, num_pages);
  if (st != LA_OK) return st;
  Pages pg{block_table, pages_per_seq, page_size, num_pages};
  return kv_evict(cfg, weights, key_pos, seq_lens, next_pos, budget, sink, recent, k_pool, v_pool,
                  weights_out, key_pos_out, kept_slots, new_lens, pg, workspace, workspace_bytes, stream);
}

la_status la_pbd_verify(int32_t dtype, const void* p, int64_t p_batch_stride, int64_t p_row_stride,
                        const void* q, int64_t q_batch_stride, int64_t q_row_stride,
                        const int32_t* drafts, const int32_t* draft_lens, const float* u,
                        const float* sample_u, int32_t batch, int32_t num_drafts, int32_t vocab,
                        int32_t* tokens, int32_t* accepted, const int32_t* seq_lens,
                        int32_t* seq_lens_out, void* stream) {
  if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_F16) return LA_ERR_INVALID_ARG;
  if (batch < 1 || num_drafts < 0 || vocab < 1) return LA_ERR_INVALID_ARG;
  if (batch > la::kMaxBatch || num_drafts > kMaxDrafts || vocab > (1 << 24)) return LA_ERR_UNSUPPORTED;
  const uintptr_t es = dtype == LA_DTYPE_F32 ? 4 : 2;
  if (!p || !sample_u || !tokens || !accepted || (num_drafts > 0 && (!drafts || !u)))
    return LA_ERR_INVALID_ARG;
  if (!aligned(p, es) || !aligned(q, es) || !aligned(drafts, 4) || !aligned(draft_lens, 4) ||
      !aligned(u, 4) || !aligned(sample_u, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) ||
      !aligned(seq_lens, 4) || !aligned(seq_lens_out, 4))
    return LA_ERR_INVALID_ARG;
  if ((seq_lens == nullptr) != (seq_lens_out == nullptr)) return LA_ERR_INVALID_ARG;
  if (p_batch_stride < 0 || p_row_stride < 0 || q_batch_stride < 0 || q_row_stride < 0)
    return LA_ERR_INVALID_ARG;
  int sms = 0;
  if (la::sm_count(&sms) != cudaSuccess) return LA_ERR_CUDA;
  la::VerifyProblem a;
  std::memset(&a, 0, sizeof(a));
  a.p = p;
  a.q = num_drafts > 0 ? q : nullptr;
  a.p_batch = p_batch_stride;
  a.p_row = p_row_stride;
  a.q_batch = q_batch_stride;
  a.q_row = q_row_stride;
  a.drafts = drafts;
  a.draft_lens = draft_lens;
  a.seq_lens = seq_lens;
  a.u = u;
  a.sample_u = sample_u;
  a.tokens = tokens;
  a.accepted = accepted;
  a.seq_lens_out = seq_lens_out;
  a.B = batch;
  a.K = num_drafts;
  a.V = vocab;
  return la::launch_verify(a, dtype, sms, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
