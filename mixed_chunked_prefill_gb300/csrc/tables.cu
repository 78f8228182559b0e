// Block tables, slot map and pages of a step, built on the GPU from request
// lengths, and the commit that moves the requests on.
//
// [L] 4.1 / 4.2 (block tables, physical address translation) and [W]
// "输入组装" (slot_mapping): what mcp_build_slot_mapping and a host allocator
// compute from host arrays, computed where the page table of every request
// already is, so that a step uploads two integers per segment.
//
// With held = ceil(len / P) and after = ceil((len + q) / P) per segment, K =
// sum(after - held): the step takes the K pages on top of the free list, in
// segment order (free[count - K + k] is new page k).  cu_seqlens_q, the new
// pages' offsets and the sampled rows are prefix sums over the segments.
//
// Work: 12 bytes per segment, 4 per held page (read) and per table entry
// (written), 12 per token slot: a few MB at most, so latency bounds every
// ordinary step (1024 segments with contexts up to 32768: 9.1 us, of which the
// bytes are 1.9).  One launch: every CTA computes the prefix sums of all
// segments for itself (two dependent loads and one block scan; S <= 8192
// segments are 4 x 32 KB of shared memory), and its warps then write their share
// of the table rows and token slots.  A second launch that waited for the sums
// would cost more than repeating them.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

constexpr int kUnit = 512;         // table entries of one row that a warp takes at a time
constexpr int kTokenUnit = 128;    // token slots that a warp takes at a time
constexpr int kWindow = 1 << 15;   // request rows per pass of the repeated-row check

struct StepArgs {
  const int32_t* ids;
  const int32_t* q_lens;
  const int32_t* new_lens;   // commit: lengths afterwards (NULL: every token stays)
  int32_t* request_pages;    // [R, width]
  int32_t* request_lens;     // [R]
  int32_t* free_pages;       // [num_pages]
  int32_t* free_count;       // [1]
  int32_t S, R, width, P_log2, num_pages, max_tokens;
  int32_t* cu;
  int32_t* sk;
  int32_t* bt;
  int64_t* slots;
  int32_t* pos;
  int32_t* rows;
  int32_t* err;
};

// Shared memory of a step: per segment the first token, the first new page
// (or, for a commit, the first returned page), the request row (-1 padding)
// and the tokens held.
struct Step {
  int32_t* cu;     // [S + 1]
  int32_t* page;   // [S + 1]
  int32_t* id;     // [S]
  int32_t* have;   // [S]
  uint32_t* seen;  // [kWindow / 32]
  int32_t base;    // free[base] is the step's first new page
  int32_t bad;     // error bits, 0: the step is sound
};

__device__ __forceinline__ int32_t pages_of(int32_t tokens, int lg) {
  return static_cast<int32_t>((static_cast<int64_t>(tokens) + (1 << lg) - 1) >> lg);
}

// Read the step's segments into shared memory, check them and scan.  Every
// CTA does the same and comes to the same answer.  A thread owns consecutive
// segments from its first load to their prefix sums, so one barrier before (the
// cleared marks), one inside the scan and one after are all.  kCommit: `page`
// receives the offsets of the returned pages.  `rows` (build, one CTA): the
// logits indices, which are one more prefix sum.
template <int kThreads, bool kCommit>
__device__ __forceinline__ void load_step(const StepArgs& p, Step& st, char* smem, int32_t* rows) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t w_tok[kWarps], w_page[kWarps], w_need[kWarps];
  __shared__ int32_t w_some[kWarps], w_bad[kWarps];
  const int32_t S = p.S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  st.cu = reinterpret_cast<int32_t*>(smem);
  st.page = st.cu + S + 1;
  st.id = st.page + S + 1;
  st.have = st.id + S;
  st.seen = reinterpret_cast<uint32_t*>(st.have + S);
  int per = (S + kThreads - 1) / kThreads;
  if (per >= 4) per |= 1;  // neighbouring threads in different banks (8000 segments: 23 us, 16 each 35)
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  const int32_t count = *p.free_count;
  const int32_t words = (min(kWindow, p.R) + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kThreads) st.seen[i] = 0;
  __syncthreads();
  const int64_t most = static_cast<int64_t>(p.width) << p.P_log2;
  int bad = count < 0 || count > p.num_pages ? MCP_DEVERR_NO_PAGES : 0;
  int64_t tok = 0, page = 0, need = 0;
  int32_t some = 0;
  for (int s = s0; s < s1; ++s) {
    const int32_t id = p.ids[s];
    int32_t q = p.q_lens[s], have = 0, back = 0, grow = 0;
    if (id < 0) {
      q = 0;  // padding: an empty segment
    } else if (id >= p.R) {
      bad |= MCP_DEVERR_REQUEST;
      q = 0;
    } else {
      have = p.request_lens[id];
      if (have < 0 || q < 0 || static_cast<int64_t>(have) + q > most) {
        bad |= MCP_DEVERR_REQUEST;
        q = have = 0;
      }
      const int32_t after = pages_of(have + q, p.P_log2);
      grow = after - pages_of(have, p.P_log2);
      if (kCommit) {
        const int32_t to = p.new_lens ? p.new_lens[s] : have + q;
        if (to < 0 || to > have + q) bad |= MCP_DEVERR_REQUEST;
        else back = after - pages_of(to, p.P_log2);
      }
      // a request may stand once in a step
      if (id < kWindow) {
        const uint32_t bit = 1u << (id & 31);
        if (atomicOr(st.seen + (id >> 5), bit) & bit) bad |= MCP_DEVERR_REQUEST;
      }
    }
    st.cu[s] = q;
    st.page[s] = kCommit ? back : grow;
    st.id[s] = id;
    st.have[s] = have;
    tok += q;
    page += kCommit ? back : grow;
    need += grow;
    some += q > 0;
  }
  for (int32_t r0 = kWindow; r0 < p.R; r0 += kWindow) {  // the other rows, a window at a time
    __syncthreads();
    for (int i = threadIdx.x; i < kWindow / 32; i += kThreads) st.seen[i] = 0;
    __syncthreads();
    for (int s = s0; s < s1; ++s) {
      const int32_t r = st.id[s] - r0;
      if (r < 0 || r >= kWindow || st.id[s] >= p.R) continue;
      const uint32_t bit = 1u << (r & 31);
      if (atomicOr(st.seen + (r >> 5), bit) & bit) bad |= MCP_DEVERR_REQUEST;
    }
  }
  const int64_t tok0 = tok, page0 = page;
  const int32_t some0 = some;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, tok, d), y = __shfl_up_sync(0xffffffffu, page, d);
    const int32_t z = __shfl_up_sync(0xffffffffu, some, d);
    if (lane >= d) tok += x, page += y, some += z;
    need += __shfl_xor_sync(0xffffffffu, need, d);
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 31) {
    w_tok[warp] = tok;
    w_page[warp] = page;
    w_some[warp] = some;
    w_need[warp] = need;
    w_bad[warp] = bad;
  }
  __syncthreads();
  tok -= tok0;
  page -= page0;
  some -= some0;
  int64_t all_tok = 0, all_page = 0, all_need = 0;
  int32_t all_some = 0;
  bad = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) tok += w_tok[w], page += w_page[w], some += w_some[w];
    all_tok += w_tok[w];
    all_page += w_page[w];
    all_some += w_some[w];
    all_need += w_need[w];
    bad |= w_bad[w];
  }
  if (all_need > count) bad |= MCP_DEVERR_NO_PAGES;
  if (kCommit && count - all_need + all_page > p.num_pages) bad |= MCP_DEVERR_NO_PAGES;
  if (all_tok > p.max_tokens) bad |= MCP_DEVERR_REQUEST;
  st.bad = bad;
  st.base = bad ? count : count - static_cast<int32_t>(all_need);
  for (int s = s0; s < s1; ++s) {
    // of an unsound step every segment is empty: nothing is taken
    const int32_t q = bad ? 0 : st.cu[s], n = bad ? 0 : st.page[s];
    if (bad) st.id[s] = -1, st.have[s] = 0, tok = page = 0;
    st.cu[s] = static_cast<int32_t>(tok);
    st.page[s] = static_cast<int32_t>(page);
    tok += q;
    page += n;
    if (rows && q > 0) rows[some++] = static_cast<int32_t>(tok) - 1;
  }
  if (threadIdx.x == 0) {
    st.cu[S] = bad ? 0 : static_cast<int32_t>(all_tok);
    st.page[S] = bad ? 0 : static_cast<int32_t>(all_page);
  }
  if (rows)
    for (int s = (bad ? 0 : all_some) + threadIdx.x; s < S; s += kThreads) rows[s] = -1;
  __syncthreads();
}

// Entry j of segment s's table row: a held page, a new page, or -1.
__device__ __forceinline__ int32_t table_entry(const int32_t* row, int32_t j, int32_t held,
                                               int32_t after, const int32_t* fresh) {
  if (j < held) return row[j];
  return j < after ? fresh[j - held] : -1;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) build_tables_kernel(const StepArgs p) {
  extern __shared__ char smem[];
  Step st;
  load_step<kThreads, false>(p, st, smem, blockIdx.x == 0 ? p.rows : nullptr);
  const int32_t S = p.S, lg = p.P_log2, width = p.width;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0 && st.bad && p.err) atomicOr(p.err, st.bad);
    for (int s = threadIdx.x; s <= S; s += kThreads) {
      p.cu[s] = st.cu[s];
      if (s < S) p.sk[s] = st.have[s] + st.cu[s + 1] - st.cu[s];
    }
  }
  // the warps of all CTAs deal out the tables' units and then the tokens'
  const int32_t per_row = (width + kUnit - 1) / kUnit;
  const int64_t tables = static_cast<int64_t>(S) * per_row;
  const int64_t units = tables + (p.max_tokens + kTokenUnit - 1) / kTokenUnit;
  const bool vec = (width & 3) == 0;  // rows 16-byte aligned
  for (int64_t u = blockIdx.x + static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x; u < units;
       u += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
    if (u < tables) {
      const int32_t s = static_cast<int32_t>(u / per_row);
      const int32_t j0 = static_cast<int32_t>(u - static_cast<int64_t>(s) * per_row) * kUnit;
      const int32_t j1 = min(width, j0 + kUnit);
      const int32_t id = st.id[s];
      const int32_t held = pages_of(st.have[s], lg);
      const int32_t after = pages_of(st.have[s] + st.cu[s + 1] - st.cu[s], lg);
      int32_t* row = p.request_pages + static_cast<int64_t>(id < 0 ? 0 : id) * width;
      const int32_t* fresh = p.free_pages + st.base + st.page[s];
      int32_t* dst = p.bt + static_cast<int64_t>(s) * width;
      if (vec) {
        constexpr int kLoads = kUnit / 128;  // in flight together
        int4 v[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int32_t j = j0 + 4 * lane + 128 * k;
          v[k] = make_int4(-1, -1, -1, -1);
          if (j + 4 <= held) v[k] = *reinterpret_cast<const int4*>(row + j);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int32_t j = j0 + 4 * lane + 128 * k;
          if (j + 4 > held && j < after) {  // the last held pages and the new ones
            v[k].x = table_entry(row, j, held, after, fresh);
            v[k].y = table_entry(row, j + 1, held, after, fresh);
            v[k].z = table_entry(row, j + 2, held, after, fresh);
            v[k].w = table_entry(row, j + 3, held, after, fresh);
          }
          if (j < j1) *reinterpret_cast<int4*>(dst + j) = v[k];
        }
      } else {
        constexpr int kLoads = kUnit / 32;
        int32_t v[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int32_t j = j0 + lane + 32 * k;
          v[k] = -1;
          if (j < held) v[k] = row[j];
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int32_t j = j0 + lane + 32 * k;
          if (j >= held && j < after) v[k] = fresh[j - held];
          if (j < j1) dst[j] = v[k];
        }
      }
      // new pages go behind the held ones (nothing else reads or writes there)
      for (int32_t j = max(j0, held) + lane; j < min(j1, after); j += 32) row[j] = fresh[j - held];
    } else {
      const int32_t t0 = static_cast<int32_t>(u - tables) * kTokenUnit;
      const int32_t T = st.cu[S];
      int lo = 0;
#pragma unroll
      for (int k = 0; k < kTokenUnit / 32; ++k) {
        const int32_t t = t0 + lane + 32 * k;
        if (t >= p.max_tokens) break;
        int64_t slot = -1;
        int32_t at = 0;
        if (t < T) {
          // the last segment that begins at or before t (it is not empty)
          if (k == 0 || st.cu[lo + 1] <= t) {
            int hi = S;
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              if (st.cu[mid] <= t) lo = mid;
              else hi = mid;
            }
          }
          at = st.have[lo] + t - st.cu[lo];
          const int32_t held = pages_of(st.have[lo], lg), j = at >> lg;
          const int32_t page = j < held
                                   ? p.request_pages[static_cast<int64_t>(st.id[lo]) * width + j]
                                   : p.free_pages[st.base + st.page[lo] + j - held];
          slot = (static_cast<int64_t>(page) << lg) + (at & ((1 << lg) - 1));
        }
        p.slots[t] = slot;
        if (p.pos) p.pos[t] = at;
      }
    }
  }
}

// Pages behind each request's new length go back to the free list; the
// lengths and the count move on.  `copy` touches only free_pages, which
// nothing here reads, and `finish` (one CTA) everything else: a launch of many
// CTAs copies, and the one that finishes may begin beside it (programmatic
// launch), as long as it writes only once all of them have read.
template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    commit_kernel(const StepArgs p, const bool copy, const bool finish) {
  extern __shared__ char smem[];
  asm volatile("griddepcontrol.launch_dependents;");
  Step st;
  load_step<kThreads, true>(p, st, smem, nullptr);
  const int32_t S = p.S, lg = p.P_log2, width = p.width;
  if (copy && !st.bad) {
    const int lane = threadIdx.x & 31;
    const int32_t per_row = (width + kUnit - 1) / kUnit;
    const int64_t units = static_cast<int64_t>(S) * per_row;
    for (int64_t u = blockIdx.x + static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x; u < units;
         u += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
      const int32_t s = static_cast<int32_t>(u / per_row);
      if (st.id[s] < 0) continue;
      const int32_t after = pages_of(st.have[s] + st.cu[s + 1] - st.cu[s], lg);
      const int32_t keep = after - (st.page[s + 1] - st.page[s]);
      const int32_t j0 = static_cast<int32_t>(u - static_cast<int64_t>(s) * per_row) * kUnit;
      const int32_t* row = p.request_pages + static_cast<int64_t>(st.id[s]) * width;
      int32_t* to = p.free_pages + st.base + st.page[s] - keep;
#pragma unroll 4
      for (int32_t j = max(j0, keep) + lane; j < min(j0 + kUnit, after); j += 32) to[j] = row[j];
    }
  }
  if (finish) {
    if (threadIdx.x == 0 && st.bad && p.err) atomicOr(p.err, st.bad);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch that copies is over
    if (st.bad) return;
    for (int s = threadIdx.x; s < S; s += kThreads) {
      if (st.id[s] < 0) continue;
      p.request_lens[st.id[s]] = p.new_lens ? p.new_lens[s] : st.have[s] + st.cu[s + 1] - st.cu[s];
    }
    if (threadIdx.x == 0) *p.free_count = st.base + st.page[S];
  }
}

size_t step_smem(int32_t S, int32_t R) {
  const int32_t window = R < kWindow ? R : kWindow;
  return (4 * static_cast<size_t>(S) + 2 + (window + 31) / 32) * 4;
}

int log2_of(int32_t v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

StepArgs step_args(const mcp_request_pool& pool, const int32_t* ids, const int32_t* q_lens,
                   int32_t S, int32_t* err) {
  StepArgs a = {};
  a.ids = ids;
  a.q_lens = q_lens;
  a.request_pages = pool.request_pages;
  a.request_lens = pool.request_lens;
  a.free_pages = pool.free_pages;
  a.free_count = pool.free_count;
  a.S = S;
  a.R = pool.max_requests;
  a.width = pool.max_pages_per_seq;
  a.P_log2 = log2_of(pool.page_size);
  a.num_pages = pool.num_pages;
  a.err = err;
  return a;
}

// CTAs for `units` warps' work, at most one per SM: each repeats the prefix sums.
int grid_of(int64_t units, int threads) {
  const int64_t ctas = (units + threads / 32 - 1) / (threads / 32), cap = step_num_sms();
  return static_cast<int>(ctas < 1 ? 1 : ctas > cap ? cap : ctas);
}

template <int kThreads>
int build_launch(const StepArgs& a, cudaStream_t st) {
  constexpr auto kernel = build_tables_kernel<kThreads>;
  if (const int e = allow_smem<kernel>(static_cast<int>(step_smem(kMaxStepSeqs, kWindow)))) return e;
  const int64_t units = static_cast<int64_t>(a.S) * ((a.width + kUnit - 1) / kUnit) +
                        (static_cast<int64_t>(a.max_tokens) + kTokenUnit - 1) / kTokenUnit;
  kernel<<<grid_of(units, kThreads), kThreads, step_smem(a.S, a.R), st>>>(a);
  return static_cast<int>(cudaGetLastError());
}

template <int kThreads>
int commit_launch(const StepArgs& a, cudaStream_t st) {
  constexpr auto kernel = commit_kernel<kThreads>;
  const size_t smem = step_smem(a.S, a.R);
  if (const int e = allow_smem<kernel>(static_cast<int>(step_smem(kMaxStepSeqs, kWindow)))) return e;
  // a commit that keeps every token returns no page: one CTA moves the lengths
  // on; it also copies what its own warps copy in two rounds
  const int64_t units = static_cast<int64_t>(a.S) * ((a.width + kUnit - 1) / kUnit);
  const bool alone = !a.new_lens || units <= 2 * kThreads / 32;
  kernel<<<alone ? 1 : grid_of(units, kThreads), kThreads, smem, st>>>(a, a.new_lens != nullptr, alone);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || alone) return static_cast<int>(e);
  return launch_beside(kernel, true, 1, kThreads, smem, st, a, false, true);
}

// Threads of a CTA: few segments are scanned faster by fewer warps (8 segments,
// build and commit: 7.1 us with 256, 8.1 with 512), many by more of them (1024
// segments of up to 32768 tokens: 9.1 us with 512, 10 with 256).
constexpr int32_t kFewSegments = 256;

}  // namespace

int step_num_sms() {
  static thread_local int dev_of = -1, sms = 152;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != dev_of) {
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    dev_of = dev;
  }
  return sms;
}

int launch_build_step_tables(const mcp_request_pool& pool, const int32_t* request_ids,
                             const int32_t* q_lens, int32_t num_seqs, int32_t max_tokens,
                             int32_t* cu_seqlens_q, int32_t* seqlens_k, int32_t* block_tables,
                             int64_t* slot_mapping, int32_t* positions, int32_t* logits_indices,
                             int32_t* error_word, void* stream) {
  StepArgs a = step_args(pool, request_ids, q_lens, num_seqs, error_word);
  a.max_tokens = max_tokens;
  a.cu = cu_seqlens_q;
  a.sk = seqlens_k;
  a.bt = block_tables;
  a.slots = slot_mapping;
  a.pos = positions;
  a.rows = logits_indices;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return num_seqs <= kFewSegments ? build_launch<256>(a, st) : build_launch<512>(a, st);
}

int launch_commit_step(const mcp_request_pool& pool, const int32_t* request_ids,
                       const int32_t* q_lens, const int32_t* new_lens, int32_t num_seqs,
                       int32_t max_tokens, int32_t* error_word, void* stream) {
  StepArgs a = step_args(pool, request_ids, q_lens, num_seqs, error_word);
  a.new_lens = new_lens;
  a.max_tokens = max_tokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return num_seqs <= kFewSegments ? commit_launch<256>(a, st) : commit_launch<512>(a, st);
}

}  // namespace mcp
