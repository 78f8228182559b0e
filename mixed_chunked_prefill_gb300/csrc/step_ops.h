// Internal declarations of the operators around a step's attention: launchers
// (return a cudaError_t value; 0 = success) called by step_ops.cpp.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mcp.h"

namespace mcp {

constexpr int32_t kMaxStepSeqs = 8192;  // segments whose prefix sums fit one CTA's shared memory

// tables.cu
int launch_build_step_tables(const mcp_request_pool& pool, const int32_t* request_ids,
                             const int32_t* q_lens, int32_t num_seqs, int32_t max_tokens,
                             int32_t* cu_seqlens_q, int32_t* seqlens_k, int32_t* block_tables,
                             int64_t* slot_mapping, int32_t* positions, int32_t* logits_indices,
                             int32_t* error_word, void* stream);
int launch_commit_step(const mcp_request_pool& pool, const int32_t* request_ids,
                       const int32_t* q_lens, const int32_t* new_lens, int32_t num_seqs,
                       int32_t max_tokens, int32_t* error_word, void* stream);
// recurrent.cu
bool mixed_conv_fits(const mcp_conv_desc& d);  // its grid is one that can be launched
int launch_mixed_conv(const mcp_conv_desc& d, const void* x, const void* weight, const void* bias,
                      void* state, const int32_t* request_ids, const int32_t* cu_seqlens_q,
                      const int32_t* seqlens_k, void* out, int32_t* error_word, void* stream);
bool mixed_scan_fits(const mcp_scan_desc& d);  // its tasks have 32-bit numbers
int launch_mixed_scan(const mcp_scan_desc& d, const mcp_scan_tensors& t,
                      const int32_t* request_ids, const int32_t* cu_seqlens_q,
                      const int32_t* seqlens_k, void* workspace, int32_t* error_word,
                      void* stream);
size_t mixed_scan_workspace(const mcp_scan_desc& d, int sms);  // bytes; 0: none is of use
// logits.cu
int launch_update_token_counts(const int32_t* request_ids, int32_t num_rows,
                               const int32_t* tokens, int32_t num_tokens,
                               const int32_t* cu_tokens, int32_t* seen, int32_t* counts,
                               int32_t num_requests, int32_t vocab_size, int32_t flags,
                               int32_t* error_word, void* stream);
int launch_process_logits(const mcp_logits_desc& d, const mcp_logits_tensors& t,
                          int32_t* error_word, void* stream);
// tree.cu
constexpr int32_t kMaxMaskWords = 32;   // a tree's rows fit one CTA's shared memory
constexpr int32_t kMaxKeepLayers = 1024;
int launch_build_tree_masks(const int32_t* parents, const int32_t* cu_seqlens_q,
                            const int32_t* seqlens_k, const int32_t* mask_rows, int32_t num_seqs,
                            int32_t total_tokens, int32_t num_mask_rows, int32_t mask_words,
                            int32_t* tree_mask, int32_t* positions, int32_t* error_word,
                            void* stream);
int launch_kv_keep_path(const mcp_keep_desc& d, void* const* k_caches, void* const* v_caches,
                        const int32_t* block_tables, const int32_t* cu_seqlens_q,
                        const int32_t* seqlens_k, const int32_t* cu_rows, const int32_t* accepted,
                        const int32_t* path, int32_t* new_lens, int32_t* error_word, void* stream);
// verify.cu
int launch_verify_drafts(const mcp_verify_desc& d, const mcp_verify_tensors& t, int32_t* error_word,
                         void* stream);

// SMs of the current device (read once per device and thread).
int step_num_sms();

// Launch a kernel that may begin beside the launch before it on the stream
// (`beside`: programmatic stream serialization).  It must not touch what that
// launch writes before its griddepcontrol.wait, and must come to that wait, so
// that what follows on the stream follows both.  0 or a cudaError_t value.
template <typename... P>
int launch_beside(void (*kernel)(P...), bool beside, int64_t grid, int block, size_t smem, cudaStream_t st,
                  const P&... args) {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &a;
  cfg.numAttrs = beside ? 1 : 0;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Allow `kernel` up to `bytes` of dynamic shared memory on the current device,
// the same `bytes` in every call (done once per device: the attribute stays).
// 0 or a cudaError_t value.
template <auto kernel>
int allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return 0;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return static_cast<int>(e);
}

}  // namespace mcp
