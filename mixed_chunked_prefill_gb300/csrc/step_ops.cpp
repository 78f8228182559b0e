// C entries of the operators around a step's attention: argument checks and
// launches (tables.cu, recurrent.cu, logits.cu, tree.cu, verify.cu).
#include "step_ops.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "mcp.h"
#include "mcp_internal.h"

namespace {

mcp_status fail(mcp_status s, const char* fmt, ...) {
  char msg[384];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return static_cast<mcp_status>(mcp::set_error_code(s, msg));
}

mcp_status done(int e, const char* what) {
  if (e != 0) return fail(MCP_ERR_CUDA, "%s: %s", what, cudaGetErrorString(static_cast<cudaError_t>(e)));
  return static_cast<mcp_status>(mcp::set_error_code(MCP_OK, ""));
}

// Sizes up to which the kernels' 32-bit indices cannot overflow (a launch rounds
// them up to its tiles).
constexpr int32_t kMaxTokens = 1 << 30;   // of a step, a stream, a list
constexpr int32_t kMaxRow = 1 << 28;      // entries of a table row, tokens of a vocabulary
constexpr int32_t kMaxRows = 1 << 24;     // request rows
constexpr int32_t kMaxSegments = 1 << 20;
constexpr int32_t kMaxChannels = 1 << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// int32 and fp32 arrays (NULL: one that is left out)
mcp_status check_words(std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned(p, 4)) return fail(MCP_ERR_INVALID_ARG, "an int32 or fp32 array is not 4-byte aligned");
  return MCP_OK;
}

// An array that a call reads or writes (NULL: none)
struct Span {
  const void* at;
  unsigned __int128 bytes;  // rows times a stride
};
Span words(const void* at, int64_t n) { return {at, static_cast<unsigned __int128>(n) * 4}; }

// The first CTA of a segment writes results while the others still read, and where CTAs
// exchange sums they have to take the same steps: a result may not be an input, nor two
// results one.
mcp_status check_apart(std::initializer_list<Span> results, std::initializer_list<Span> inputs) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x && y && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
  };
  for (const Span* r = results.begin(); r != results.end(); ++r) {
    for (const Span& i : inputs)
      if (meet(*r, i)) return fail(MCP_ERR_INVALID_ARG, "a result may not overlap an input");
    for (const Span* q = results.begin(); q != r; ++q)
      if (meet(*r, *q)) return fail(MCP_ERR_INVALID_ARG, "results may not overlap each other");
  }
  return MCP_OK;
}

// Whether two of the caches of a call to mcp_kv_keep_path share memory: rows move in place, so a
// cache that stands for two layers, or for K and V, would move its rows twice.
bool caches_overlap(const mcp_keep_desc& d, void* const* k, void* const* v) {
  using Wide = __int128;
  const Wide bytes = static_cast<Wide>(d.num_pages) * d.page_size * d.num_kv_heads * d.head_dim * 2;
  const int32_t L = d.num_layers;
  if (L == 0) return false;
  if (d.layer_stride != 0) {
    const Wide step = static_cast<Wide>(d.layer_stride) * 2;
    if (L > 1 && step < bytes) return true;
    const Wide apart = static_cast<Wide>(reinterpret_cast<uintptr_t>(v[0])) - reinterpret_cast<uintptr_t>(k[0]);
    // V of layer l lies apart + (l - m) step behind K of layer m: the nearest of these
    const Wide near = L > 1 ? -apart / step : 0;
    for (Wide j = near - 1; j <= near + 1; ++j)
      if (j > -L && j < L && apart + j * step < bytes && apart + j * step > -bytes) return true;
    return false;
  }
  uintptr_t at[2 * mcp::kMaxKeepLayers];
  for (int32_t l = 0; l < L; ++l) {
    at[2 * l] = reinterpret_cast<uintptr_t>(k[l]);
    at[2 * l + 1] = reinterpret_cast<uintptr_t>(v[l]);
  }
  std::sort(at, at + 2 * L);
  for (int32_t i = 1; i < 2 * L; ++i)
    if (at[i] - at[i - 1] < bytes) return true;
  return false;
}

#define MCP_TRY(expr)                    \
  do {                                   \
    const mcp_status st_ = (expr);       \
    if (st_ != MCP_OK) return st_;       \
  } while (0)

mcp_status check_pool(const mcp_request_pool* p, int32_t num_seqs, const int32_t* ids,
                      const int32_t* q_lens) {
  if (!p) return fail(MCP_ERR_INVALID_ARG, "pool is NULL");
  if (num_seqs < 0) return fail(MCP_ERR_INVALID_ARG, "num_seqs %d < 0", num_seqs);
  if (num_seqs > mcp::kMaxStepSeqs)
    return fail(MCP_ERR_UNSUPPORTED, "num_seqs %d > %d", num_seqs, mcp::kMaxStepSeqs);
  if (p->max_requests <= 0 || p->max_pages_per_seq <= 0 || p->num_pages <= 0)
    return fail(MCP_ERR_INVALID_ARG, "pool sizes must be positive (requests %d, row %d, pages %d)",
                p->max_requests, p->max_pages_per_seq, p->num_pages);
  if (p->max_requests > kMaxRows || p->max_pages_per_seq > kMaxRow)
    return fail(MCP_ERR_UNSUPPORTED, "max_requests %d > 2^24 or max_pages_per_seq %d > 2^28", p->max_requests,
                p->max_pages_per_seq);
  if (p->page_size != 1 && p->page_size != 8 && p->page_size != 16 && p->page_size != 32 &&
      p->page_size != 64)
    return fail(MCP_ERR_UNSUPPORTED, "page_size %d (built: 1, 8, 16, 32, 64)", p->page_size);
  if (static_cast<int64_t>(p->max_pages_per_seq) * p->page_size > 0x7fffffff)
    return fail(MCP_ERR_UNSUPPORTED, "max_pages_per_seq * page_size must be below 2^31");
  if (!p->request_pages || !p->request_lens || !p->free_pages || !p->free_count)
    return fail(MCP_ERR_INVALID_ARG, "NULL pointer in the pool");
  if (!aligned(p->request_pages, 16) || !aligned(p->request_lens, 4) || !aligned(p->free_pages, 4) ||
      !aligned(p->free_count, 4))
    return fail(MCP_ERR_INVALID_ARG, "pool tensor misaligned (request_pages: 16 bytes)");
  if (num_seqs > 0 && (!ids || !q_lens)) return fail(MCP_ERR_INVALID_ARG, "NULL pointer argument");
  return check_words({ids, q_lens});
}

mcp_status check_max_tokens(int32_t max_tokens) {
  if (max_tokens < 0) return fail(MCP_ERR_INVALID_ARG, "max_tokens %d < 0", max_tokens);
  if (max_tokens > kMaxTokens) return fail(MCP_ERR_UNSUPPORTED, "max_tokens %d > 2^30", max_tokens);
  return MCP_OK;
}

mcp_status check_stream_sizes(int32_t num_seqs, int32_t tokens, int32_t requests, int32_t channels,
                              int32_t dtype) {
  if (num_seqs < 0 || tokens < 0)
    return fail(MCP_ERR_INVALID_ARG, "num_seqs %d / total_tokens %d < 0", num_seqs, tokens);
  if (requests <= 0 || channels <= 0)
    return fail(MCP_ERR_INVALID_ARG, "num_requests %d / channels %d must be positive", requests,
                channels);
  if (num_seqs > kMaxSegments || tokens > kMaxTokens || requests > kMaxRows || channels > kMaxChannels)
    return fail(MCP_ERR_UNSUPPORTED,
                "num_seqs %d > 2^20, total_tokens %d > 2^30, num_requests %d > 2^24 or channels %d > 2^30",
                num_seqs, tokens, requests, channels);
  if (channels % 8 != 0)
    return fail(MCP_ERR_INVALID_ARG, "channels %d is not a multiple of 8", channels);
  if (dtype != MCP_DTYPE_BF16 && dtype != MCP_DTYPE_FP16)
    return fail(MCP_ERR_UNSUPPORTED, "dtype %d (built: bf16, fp16)", dtype);
  return MCP_OK;
}

// `t` [tokens, row] with `stride` elements between tokens
mcp_status check_rows(const void* t, int64_t stride, int64_t row, const char* name) {
  if (!t) return fail(MCP_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(t, 16)) return fail(MCP_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < row || stride % 8 != 0)
    return fail(MCP_ERR_INVALID_ARG, "%s: token stride %lld must be a multiple of 8 and >= %lld", name,
                static_cast<long long>(stride), static_cast<long long>(row));
  return MCP_OK;
}

mcp_status check_scan_desc(const mcp_scan_desc* d) {
  if (!d) return fail(MCP_ERR_INVALID_ARG, "desc is NULL");
  MCP_TRY(check_stream_sizes(d->num_seqs, d->total_tokens, d->num_requests, d->channels, d->dtype));
  if (d->state_size != 8 && d->state_size != 16 && d->state_size != 32 && d->state_size != 64)
    return fail(MCP_ERR_UNSUPPORTED, "state_size %d (built: 8, 16, 32, 64)", d->state_size);
  if (d->num_groups <= 0 || d->channels % d->num_groups != 0)
    return fail(MCP_ERR_INVALID_ARG, "num_groups %d does not divide channels %d", d->num_groups,
                d->channels);
  if (d->num_groups > 1 && d->channels / d->num_groups % 32 != 0)
    return fail(MCP_ERR_UNSUPPORTED, "%d channels a group (built: multiples of 32)",
                d->channels / d->num_groups);
  if (d->softplus != 0 && d->softplus != 1)
    return fail(MCP_ERR_INVALID_ARG, "softplus %d (0 or 1)", d->softplus);
  return MCP_OK;
}

}  // namespace

extern "C" {

mcp_status mcp_build_step_tables(const mcp_request_pool* pool, const int32_t* request_ids,
                                 const int32_t* q_lens, int32_t num_seqs, int32_t max_tokens,
                                 int32_t* cu_seqlens_q, int32_t* seqlens_k, int32_t* block_tables,
                                 int64_t* slot_mapping, int32_t* positions,
                                 int32_t* logits_indices, int32_t* error_word, void* stream) {
  MCP_TRY(check_pool(pool, num_seqs, request_ids, q_lens));
  MCP_TRY(check_max_tokens(max_tokens));
  if (!cu_seqlens_q || (num_seqs > 0 && (!seqlens_k || !block_tables)) ||
      (max_tokens > 0 && !slot_mapping))
    return fail(MCP_ERR_INVALID_ARG, "NULL output pointer");
  if (!aligned(block_tables, 16) || !aligned(slot_mapping, 8))
    return fail(MCP_ERR_INVALID_ARG, "block_tables must be 16-byte, slot_mapping 8-byte aligned");
  MCP_TRY(check_words({cu_seqlens_q, seqlens_k, positions, logits_indices, error_word}));
  return done(mcp::launch_build_step_tables(*pool, request_ids, q_lens, num_seqs, max_tokens,
                                            cu_seqlens_q, seqlens_k, block_tables, slot_mapping,
                                            positions, logits_indices, error_word, stream),
              "build_step_tables launch");
}

mcp_status mcp_commit_step(const mcp_request_pool* pool, const int32_t* request_ids,
                           const int32_t* q_lens, const int32_t* new_lens, int32_t num_seqs,
                           int32_t* error_word, void* stream) {
  return mcp_commit_built_step(pool, request_ids, q_lens, new_lens, num_seqs, kMaxTokens, error_word,
                               stream);
}

mcp_status mcp_commit_built_step(const mcp_request_pool* pool, const int32_t* request_ids,
                                 const int32_t* q_lens, const int32_t* new_lens, int32_t num_seqs,
                                 int32_t max_tokens, int32_t* error_word, void* stream) {
  MCP_TRY(check_pool(pool, num_seqs, request_ids, q_lens));
  MCP_TRY(check_max_tokens(max_tokens));
  MCP_TRY(check_words({new_lens, error_word}));
  if (num_seqs == 0) return done(0, "");
  return done(mcp::launch_commit_step(*pool, request_ids, q_lens, new_lens, num_seqs, max_tokens,
                                      error_word, stream),
              "commit_step launch");
}

mcp_status mcp_mixed_conv(const mcp_conv_desc* d, const void* x, const void* weight,
                          const void* bias, void* state, const int32_t* request_ids,
                          const int32_t* cu_seqlens_q, const int32_t* seqlens_k, void* out,
                          int32_t* error_word, void* stream) {
  if (!d) return fail(MCP_ERR_INVALID_ARG, "desc is NULL");
  MCP_TRY(check_stream_sizes(d->num_seqs, d->total_tokens, d->num_requests, d->channels, d->dtype));
  if (d->num_seqs > 0 && (!request_ids || !cu_seqlens_q || !seqlens_k))
    return fail(MCP_ERR_INVALID_ARG, "NULL metadata pointer");
  MCP_TRY(check_words({request_ids, cu_seqlens_q, seqlens_k, error_word}));
  if (d->width < 2 || d->width > 4)
    return fail(MCP_ERR_UNSUPPORTED, "width %d (built: 2, 3, 4)", d->width);
  if (d->activation != 0 && d->activation != 1)
    return fail(MCP_ERR_INVALID_ARG, "activation %d (0 none, 1 silu)", d->activation);
  if (d->reserved != 0) return fail(MCP_ERR_INVALID_ARG, "reserved fields must be 0");
  if (d->num_seqs == 0 || d->total_tokens == 0) return done(0, "");
  MCP_TRY(check_rows(x, d->x_stride, d->channels, "x"));
  MCP_TRY(check_rows(out, d->out_stride, d->channels, "out"));
  if (!weight || !state) return fail(MCP_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned(weight, 16) || !aligned(bias, 16) || !aligned(state, 16))
    return fail(MCP_ERR_INVALID_ARG, "weight, bias and state must be 16-byte aligned");
  if (out == x) return fail(MCP_ERR_INVALID_ARG, "out may not overlap x (a token reads those before it)");
  if (!mcp::mixed_conv_fits(*d))
    return fail(MCP_ERR_UNSUPPORTED, "num_seqs %d, total_tokens %d and channels %d exceed a launch", d->num_seqs,
                d->total_tokens, d->channels);
  return done(mcp::launch_mixed_conv(*d, x, weight, bias, state, request_ids, cu_seqlens_q, seqlens_k,
                                     out, error_word, stream),
              "mixed_conv launch");
}

mcp_status mcp_mixed_scan_workspace(const mcp_scan_desc* d, size_t* workspace_bytes) {
  if (!workspace_bytes) return fail(MCP_ERR_INVALID_ARG, "workspace_bytes is NULL");
  MCP_TRY(check_scan_desc(d));
  *workspace_bytes = mcp::mixed_scan_workspace(*d, mcp::step_num_sms());
  return done(0, "");
}

mcp_status mcp_mixed_scan(const mcp_scan_desc* d, const mcp_scan_tensors* t,
                          const int32_t* request_ids, const int32_t* cu_seqlens_q,
                          const int32_t* seqlens_k, void* workspace, size_t workspace_bytes,
                          int32_t* error_word, void* stream) {
  MCP_TRY(check_scan_desc(d));
  if (!t) return fail(MCP_ERR_INVALID_ARG, "tensors is NULL");
  if (d->num_seqs > 0 && (!request_ids || !cu_seqlens_q || !seqlens_k))
    return fail(MCP_ERR_INVALID_ARG, "NULL metadata pointer");
  MCP_TRY(check_words({request_ids, cu_seqlens_q, seqlens_k, error_word}));
  if (d->num_seqs == 0 || d->total_tokens == 0) return done(0, "");
  const int64_t gn = static_cast<int64_t>(d->num_groups) * d->state_size;
  MCP_TRY(check_rows(t->x, d->x_stride, d->channels, "x"));
  MCP_TRY(check_rows(t->dt, d->dt_stride, d->channels, "dt"));
  MCP_TRY(check_rows(t->B, d->b_stride, gn, "B"));
  MCP_TRY(check_rows(t->C, d->c_stride, gn, "C"));
  if (t->z) MCP_TRY(check_rows(t->z, d->z_stride, d->channels, "z"));
  MCP_TRY(check_rows(t->out, d->out_stride, d->channels, "out"));
  if (!t->A || !t->state) return fail(MCP_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned(t->A, 16) || !aligned(t->state, 16) || !aligned(t->D, 16) || !aligned(t->dt_bias, 16))
    return fail(MCP_ERR_INVALID_ARG, "A, D, dt_bias and state must be 16-byte aligned");
  if (workspace) {
    if (!aligned(workspace, 256)) return fail(MCP_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    const size_t need = mcp::mixed_scan_workspace(*d, mcp::step_num_sms());
    if (workspace_bytes < need)
      return fail(MCP_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, %zu needed", workspace_bytes, need);
  }
  for (const void* in : {t->x, t->dt, t->B, t->C, t->z})
    if (t->out == in) return fail(MCP_ERR_INVALID_ARG, "out may not overlap an input");
  if (!mcp::mixed_scan_fits(*d))
    return fail(MCP_ERR_UNSUPPORTED, "num_seqs %d, total_tokens %d and channels %d exceed a launch", d->num_seqs,
                d->total_tokens, d->channels);
  return done(mcp::launch_mixed_scan(*d, *t, request_ids, cu_seqlens_q, seqlens_k, workspace,
                                     error_word, stream),
              "mixed_scan launch");
}

mcp_status mcp_update_token_counts(const int32_t* request_ids, int32_t num_rows,
                                   const int32_t* tokens, int32_t num_tokens,
                                   const int32_t* cu_tokens, int32_t* seen, int32_t* counts,
                                   int32_t num_requests, int32_t vocab_size, int32_t flags,
                                   int32_t* error_word, void* stream) {
  if (num_rows < 0 || num_tokens < 0)
    return fail(MCP_ERR_INVALID_ARG, "num_rows %d / num_tokens %d < 0", num_rows, num_tokens);
  if (num_requests <= 0 || vocab_size <= 0)
    return fail(MCP_ERR_INVALID_ARG, "num_requests %d / vocab_size %d must be positive", num_requests,
                vocab_size);
  if (num_tokens > kMaxTokens || num_rows > kMaxTokens || vocab_size > kMaxRow)
    return fail(MCP_ERR_UNSUPPORTED, "num_tokens %d or num_rows %d > 2^30, or vocab_size %d > 2^28", num_tokens,
                num_rows, vocab_size);
  if (flags & ~(MCP_COUNT_PROMPT | MCP_COUNT_RESET))
    return fail(MCP_ERR_INVALID_ARG, "flags 0x%x", flags);
  if (!cu_tokens && num_tokens != num_rows)
    return fail(MCP_ERR_INVALID_ARG, "%d tokens for %d rows without cu_tokens", num_tokens, num_rows);
  if (num_rows == 0) return done(0, "");
  if (!request_ids || !seen || !counts || (num_tokens > 0 && !tokens))
    return fail(MCP_ERR_INVALID_ARG, "NULL tensor pointer");
  MCP_TRY(check_words({request_ids, tokens, cu_tokens, seen, counts, error_word}));
  return done(mcp::launch_update_token_counts(request_ids, num_rows, tokens, num_tokens, cu_tokens,
                                              seen, counts, num_requests, vocab_size, flags,
                                              error_word, stream),
              "update_token_counts launch");
}

mcp_status mcp_process_logits(const mcp_logits_desc* d, const mcp_logits_tensors* t,
                              int32_t* error_word, void* stream) {
  if (!d || !t) return fail(MCP_ERR_INVALID_ARG, "desc or tensors is NULL");
  if (d->num_rows < 0 || d->vocab_size <= 0)
    return fail(MCP_ERR_INVALID_ARG, "num_rows %d / vocab_size %d", d->num_rows, d->vocab_size);
  if (d->vocab_size > kMaxRow) return fail(MCP_ERR_UNSUPPORTED, "vocab_size %d > 2^28", d->vocab_size);
  if (d->dtype != MCP_DTYPE_BF16 && d->dtype != MCP_DTYPE_FP16 && d->dtype != MCP_DTYPE_FP32)
    return fail(MCP_ERR_UNSUPPORTED, "dtype %d", d->dtype);
  if (d->out_dtype != d->dtype && d->out_dtype != MCP_DTYPE_FP32)
    return fail(MCP_ERR_UNSUPPORTED, "out_dtype %d (built: the logits' type, fp32)", d->out_dtype);
  if (d->reserved != 0) return fail(MCP_ERR_INVALID_ARG, "reserved fields must be 0");
  if (d->logits_stride < d->vocab_size || d->out_stride < d->vocab_size)
    return fail(MCP_ERR_INVALID_ARG, "row stride below vocab_size %d", d->vocab_size);
  if (static_cast<int64_t>(d->num_rows) * ((d->vocab_size + 2047LL) / 2048) > 0x7fffffff)
    return fail(MCP_ERR_UNSUPPORTED, "num_rows %d x vocab_size %d", d->num_rows, d->vocab_size);
  if (d->num_biases < 0 || d->num_masks < 0 || d->num_requests < 0)
    return fail(MCP_ERR_INVALID_ARG, "negative count");
  if (d->num_rows == 0) return done(0, "");
  if (!t->logits || !t->out) return fail(MCP_ERR_INVALID_ARG, "logits or out is NULL");
  const uintptr_t in = d->dtype == MCP_DTYPE_FP32 ? 4 : 2, out = d->out_dtype == MCP_DTYPE_FP32 ? 4 : 2;
  if (!aligned(t->logits, in) || !aligned(t->out, out))
    return fail(MCP_ERR_INVALID_ARG, "logits or out misaligned");
  if (t->logits == t->out && (d->dtype != d->out_dtype || d->logits_stride != d->out_stride))
    return fail(MCP_ERR_INVALID_ARG, "in place needs one type and one row stride");
  if (t->request_ids && (!t->seen || !t->counts || d->num_requests == 0))
    return fail(MCP_ERR_INVALID_ARG, "request_ids without seen and counts");
  if (!t->request_ids && (t->repetition_penalty || t->frequency_penalty || t->presence_penalty))
    return fail(MCP_ERR_INVALID_ARG, "penalties need request_ids, seen and counts");
  MCP_TRY(check_words({t->request_ids, t->seen, t->temperature, t->repetition_penalty, t->frequency_penalty,
                       t->presence_penalty, t->bias_offsets, t->bias_tokens, t->bias_values, t->mask,
                       t->mask_rows, error_word}));
  if (!aligned(t->counts, 16)) return fail(MCP_ERR_INVALID_ARG, "counts must be 16-byte aligned");
  if (t->bias_offsets && d->num_biases > 0 && (!t->bias_tokens || !t->bias_values))
    return fail(MCP_ERR_INVALID_ARG, "bias_offsets without bias_tokens and bias_values");
  if (t->mask && !t->mask_rows && d->num_masks < d->num_rows)
    return fail(MCP_ERR_INVALID_ARG, "%d masks for %d rows without mask_rows", d->num_masks,
                d->num_rows);
  if (!t->mask && t->mask_rows) return fail(MCP_ERR_INVALID_ARG, "mask_rows without mask");
  return done(mcp::launch_process_logits(*d, *t, error_word, stream), "process_logits launch");
}

mcp_status mcp_build_tree_masks(const int32_t* parents, const int32_t* cu_seqlens_q,
                                const int32_t* seqlens_k, const int32_t* mask_rows,
                                int32_t num_seqs, int32_t total_tokens, int32_t num_mask_rows,
                                int32_t mask_words, int32_t* tree_mask, int32_t* positions,
                                int32_t* error_word, void* stream) {
  if (num_seqs < 0 || total_tokens < 0 || num_mask_rows < 0 || mask_words <= 0)
    return fail(MCP_ERR_INVALID_ARG, "num_seqs %d / total_tokens %d / num_mask_rows %d / mask_words %d",
                num_seqs, total_tokens, num_mask_rows, mask_words);
  if (num_seqs > kMaxSegments || total_tokens > kMaxTokens || num_mask_rows > kMaxTokens ||
      mask_words > mcp::kMaxMaskWords)
    return fail(MCP_ERR_UNSUPPORTED,
                "num_seqs %d > 2^20, total_tokens %d or num_mask_rows %d > 2^30, or mask_words %d > %d",
                num_seqs, total_tokens, num_mask_rows, mask_words, mcp::kMaxMaskWords);
  MCP_TRY(check_words({parents, cu_seqlens_q, seqlens_k, mask_rows, tree_mask, positions, error_word}));
  if (num_seqs == 0 || total_tokens == 0) return done(0, "");
  if (!parents || !cu_seqlens_q || !seqlens_k || !mask_rows || (num_mask_rows > 0 && !tree_mask))
    return fail(MCP_ERR_INVALID_ARG, "NULL pointer argument");
  MCP_TRY(check_apart({words(tree_mask, static_cast<int64_t>(num_mask_rows) * mask_words),
                       words(positions, total_tokens)},
                      {words(parents, total_tokens), words(cu_seqlens_q, num_seqs + 1),
                       words(seqlens_k, num_seqs), words(mask_rows, num_seqs), words(error_word, 1)}));
  return done(mcp::launch_build_tree_masks(parents, cu_seqlens_q, seqlens_k, mask_rows, num_seqs,
                                           total_tokens, num_mask_rows, mask_words, tree_mask,
                                           positions, error_word, stream),
              "build_tree_masks launch");
}

mcp_status mcp_verify_drafts(const mcp_verify_desc* d, const mcp_verify_tensors* t,
                             int32_t* error_word, void* stream) {
  if (!d || !t) return fail(MCP_ERR_INVALID_ARG, "desc or tensors is NULL");
  if (d->num_seqs < 0 || d->total_rows < 0 || d->vocab_size <= 0)
    return fail(MCP_ERR_INVALID_ARG, "num_seqs %d / total_rows %d / vocab_size %d", d->num_seqs,
                d->total_rows, d->vocab_size);
  if (d->num_seqs > kMaxSegments || d->total_rows > kMaxTokens || d->vocab_size > kMaxRow)
    return fail(MCP_ERR_UNSUPPORTED, "num_seqs %d > 2^20, total_rows %d > 2^30 or vocab_size %d > 2^28",
                d->num_seqs, d->total_rows, d->vocab_size);
  if (d->dtype != MCP_DTYPE_BF16 && d->dtype != MCP_DTYPE_FP16 && d->dtype != MCP_DTYPE_FP32)
    return fail(MCP_ERR_UNSUPPORTED, "dtype %d", d->dtype);
  if (d->target_stride < d->vocab_size || (t->draft && d->draft_stride < d->vocab_size))
    return fail(MCP_ERR_INVALID_ARG, "row stride below vocab_size %d", d->vocab_size);
  if (d->num_seqs == 0) return done(0, "");
  if (!t->cu_rows || !t->final_uniform || !t->accepted ||
      (d->total_rows > 0 && (!t->target || !t->tokens || !t->uniform || !t->path || !t->new_tokens)))
    return fail(MCP_ERR_INVALID_ARG, "NULL tensor pointer");
  const uintptr_t size = d->dtype == MCP_DTYPE_FP32 ? 4 : 2;
  if (!aligned(t->target, size) || !aligned(t->draft, size))
    return fail(MCP_ERR_INVALID_ARG, "target or draft misaligned");
  MCP_TRY(check_words({t->tokens, t->parents, t->cu_rows, t->uniform, t->final_uniform, t->accepted,
                       t->path, t->new_tokens, error_word}));
  auto rows = [&](const void* at, int64_t stride) {
    return Span{at, d->total_rows == 0 ? 0 : (static_cast<unsigned __int128>(d->total_rows - 1) * stride +
                                              d->vocab_size) * size};
  };
  MCP_TRY(check_apart({words(t->accepted, d->num_seqs), words(t->path, d->total_rows),
                       words(t->new_tokens, d->total_rows)},
                      {rows(t->target, d->target_stride), rows(t->draft, d->draft_stride),
                       words(t->tokens, d->total_rows), words(t->parents, d->total_rows),
                       words(t->cu_rows, d->num_seqs + 1), words(t->uniform, d->total_rows),
                       words(t->final_uniform, d->num_seqs), words(error_word, 1)}));
  return done(mcp::launch_verify_drafts(*d, *t, error_word, stream), "verify_drafts launch");
}

mcp_status mcp_kv_keep_path(const mcp_keep_desc* d, void* const* k_caches, void* const* v_caches,
                            const int32_t* block_tables, const int32_t* cu_seqlens_q,
                            const int32_t* seqlens_k, const int32_t* cu_rows,
                            const int32_t* accepted, const int32_t* path, int32_t* new_lens,
                            int32_t* error_word, void* stream) {
  if (!d) return fail(MCP_ERR_INVALID_ARG, "desc is NULL");
  if (d->num_seqs < 0 || d->total_rows < 0 || d->num_layers < 0)
    return fail(MCP_ERR_INVALID_ARG, "num_seqs %d / total_rows %d / num_layers %d < 0", d->num_seqs,
                d->total_rows, d->num_layers);
  if (d->num_seqs > kMaxSegments || d->total_rows > kMaxTokens || d->num_layers > mcp::kMaxKeepLayers)
    return fail(MCP_ERR_UNSUPPORTED, "num_seqs %d > 2^20, total_rows %d > 2^30 or num_layers %d > %d",
                d->num_seqs, d->total_rows, d->num_layers, mcp::kMaxKeepLayers);
  if (d->num_kv_heads <= 0 || d->head_dim <= 0 || d->max_pages_per_seq <= 0 || d->num_pages <= 0)
    return fail(MCP_ERR_INVALID_ARG, "sizes must be positive (heads %d, dim %d, table row %d, pages %d)",
                d->num_kv_heads, d->head_dim, d->max_pages_per_seq, d->num_pages);
  if (d->page_size != 1 && d->page_size != 8 && d->page_size != 16 && d->page_size != 32 &&
      d->page_size != 64)
    return fail(MCP_ERR_UNSUPPORTED, "page_size %d (built: 1, 8, 16, 32, 64)", d->page_size);
  const int64_t row = static_cast<int64_t>(d->num_kv_heads) * d->head_dim;
  if (row % 8 != 0)
    return fail(MCP_ERR_INVALID_ARG, "num_kv_heads * head_dim = %lld is not a multiple of 8",
                static_cast<long long>(row));
  if (row > 1 << 20 || d->max_pages_per_seq > kMaxRow)
    return fail(MCP_ERR_UNSUPPORTED, "num_kv_heads * head_dim %lld > 2^20 or max_pages_per_seq %d > 2^28",
                static_cast<long long>(row), d->max_pages_per_seq);
  MCP_TRY(check_words({block_tables, cu_seqlens_q, seqlens_k, cu_rows, accepted, path, new_lens, error_word}));
  if (d->num_seqs == 0) return done(0, "");
  if (!block_tables || !cu_seqlens_q || !seqlens_k || !accepted || (d->total_rows > 0 && !path) ||
      (d->num_layers > 0 && (!k_caches || !v_caches)))
    return fail(MCP_ERR_INVALID_ARG, "NULL pointer argument");
  if (d->layer_stride < 0 || d->layer_stride % 8 != 0)
    return fail(MCP_ERR_INVALID_ARG, "layer_stride %lld is not a multiple of 8",
                static_cast<long long>(d->layer_stride));
  for (int32_t l = 0; l < (d->layer_stride && d->num_layers ? 1 : d->num_layers); ++l)
    if (!k_caches[l] || !v_caches[l] || !aligned(k_caches[l], 16) || !aligned(v_caches[l], 16))
      return fail(MCP_ERR_INVALID_ARG, "cache of layer %d is NULL or not 16-byte aligned", l);
  MCP_TRY(check_apart({words(new_lens, d->num_seqs)},
                      {words(block_tables, static_cast<int64_t>(d->num_seqs) * d->max_pages_per_seq),
                       words(cu_seqlens_q, d->num_seqs + 1), words(seqlens_k, d->num_seqs),
                       words(cu_rows, d->num_seqs + 1), words(accepted, d->num_seqs),
                       words(path, d->total_rows), words(error_word, 1)}));
  if (caches_overlap(*d, k_caches, v_caches))
    return fail(MCP_ERR_INVALID_ARG, "caches overlap: each layer's K and V must be memory of their own");
  return done(mcp::launch_kv_keep_path(*d, k_caches, v_caches, block_tables, cu_seqlens_q, seqlens_k,
                                       cu_rows, accepted, path, new_lens, error_word, stream),
              "kv_keep_path launch");
}

}  // extern "C"
