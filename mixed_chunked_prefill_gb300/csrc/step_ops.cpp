// C entries of the operators around a step's attention: argument checks and
// launches (tables.cu, recurrent.cu, logits.cu).
#include "step_ops.h"

#include <cuda_runtime.h>

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

}  // extern "C"
