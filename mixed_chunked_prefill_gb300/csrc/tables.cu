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
// ordinary step.  One launch: every CTA computes the prefix sums of all
// segments for itself (two dependent loads and one block scan; S <= 8192
// segments are 4 x 32 KB of shared memory) and then writes its share of the
// table rows and token slots.  A second launch that waited for the sums would
// cost more than repeating them.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

constexpr int kThreads = 512;
constexpr int kPiece = 2048;       // table entries of one row, or token slots, per work piece
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
  int32_t* seen;   // [kWindow / 32]
  int32_t base;    // free[base] is the step's first new page
  int32_t count;   // free_count before the step
  int32_t bad;     // error bits, 0: the step is sound
};

__device__ __forceinline__ int32_t pages_of(int32_t tokens, int lg) {
  return static_cast<int32_t>((static_cast<int64_t>(tokens) + (1 << lg) - 1) >> lg);
}

// Exclusive block sums of a and b over the threads; totals in ta, tb.
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb) {
  __shared__ int64_t wa[kThreads / 32], wb[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t a0 = a, b0 = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) a += x, b += y;
  }
  __syncthreads();  // wa / wb may still be read from the scan before
  if (lane == 31) wa[warp] = a, wb[warp] = b;
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) pa = ta, pb = tb;
    ta += wa[w];
    tb += wb[w];
  }
  a = pa + a - a0;
  b = pb + b - b0;
}

// Read the step's segments into shared memory, check them and scan.  Every
// CTA does the same and comes to the same answer.  kCommit: `page` receives
// the offsets of the returned pages.
template <bool kCommit>
__device__ __forceinline__ void load_step(const StepArgs& p, Step& st, char* smem) {
  const int32_t S = p.S;
  st.cu = reinterpret_cast<int32_t*>(smem);
  st.page = st.cu + S + 1;
  st.id = st.page + S + 1;
  st.have = st.id + S;
  st.seen = st.have + S;
  st.count = *p.free_count;
  int bad = st.count < 0 || st.count > p.num_pages ? MCP_DEVERR_NO_PAGES : 0;
  const int64_t most = static_cast<int64_t>(p.width) << p.P_log2;
  int64_t need = 0;  // new pages of this thread's segments
  for (int s = threadIdx.x; s < S; s += kThreads) {
    const int32_t id = p.ids[s];
    int32_t q = p.q_lens[s], have = 0, back = 0, grow = 0;
    if (id < 0) {
      q = 0;  // padding: an empty segment
    } else if (id >= p.R) {
      bad |= MCP_DEVERR_REQUEST;
    } else {
      have = p.request_lens[id];
      if (have < 0 || q < 0 || static_cast<int64_t>(have) + q > most) {
        bad |= MCP_DEVERR_REQUEST;
        q = have = 0;
      }
      const int32_t after = pages_of(have + q, p.P_log2);
      grow = after - pages_of(have, p.P_log2);
      need += grow;
      if (kCommit) {
        const int32_t to = p.new_lens ? p.new_lens[s] : have + q;
        if (to < 0 || to > have + q)
          bad |= MCP_DEVERR_REQUEST;
        else
          back = after - pages_of(to, p.P_log2);
      }
    }
    st.cu[s] = q;
    st.page[s] = kCommit ? back : grow;
    st.id[s] = id;
    st.have[s] = have;
  }
  // a request may stand once in a step: mark the rows, a window at a time
  for (int32_t w0 = 0; w0 < p.R; w0 += kWindow) {
    const int32_t words = (min(kWindow, p.R - w0) + 31) / 32;
    __syncthreads();
    for (int i = threadIdx.x; i < words; i += kThreads) st.seen[i] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < S; s += kThreads) {
      const int32_t r = st.id[s] - w0;
      if (st.id[s] < 0 || r < 0 || r >= kWindow || st.id[s] >= p.R) continue;
      const int32_t bit = static_cast<int32_t>(1u << (r & 31));
      if (atomicOr(st.seen + (r >> 5), bit) & bit) bad |= MCP_DEVERR_REQUEST;
    }
  }
  __syncthreads();
  // prefix sums: each thread owns consecutive segments
  const int per = (S + kThreads - 1) / kThreads;
  const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
  int64_t a = 0, b = 0, ta, tb;
  for (int s = s0; s < s1; ++s) a += st.cu[s], b += st.page[s];
  block_scan2(a, b, ta, tb);
  int64_t total_need = tb;
  if (kCommit) {
    int64_t none = 0, nt;
    block_scan2(need, none, total_need, nt);
  }
  if (total_need > st.count) bad |= MCP_DEVERR_NO_PAGES;
  if (!kCommit && ta > p.max_tokens) bad |= MCP_DEVERR_REQUEST;
  if (kCommit && st.count - total_need + tb > p.num_pages) bad |= MCP_DEVERR_NO_PAGES;
  if (ta > 0x7fffffff) bad |= MCP_DEVERR_REQUEST;
  // the error bits of all threads (two bits in use)
  const int no_pages = __syncthreads_or(bad & MCP_DEVERR_NO_PAGES);
  const int request = __syncthreads_or(bad & MCP_DEVERR_REQUEST);
  st.bad = (no_pages ? MCP_DEVERR_NO_PAGES : 0) | (request ? MCP_DEVERR_REQUEST : 0);
  st.base = st.count - static_cast<int32_t>(st.bad ? 0 : total_need);
  if (st.bad) {
    // an empty step: nothing is taken, every segment without tokens or pages
    a = b = ta = tb = 0;
    for (int s = s0; s < s1; ++s) st.cu[s] = st.page[s] = st.have[s] = 0, st.id[s] = -1;
  }
  for (int s = s0; s < s1; ++s) {
    const int32_t q = st.cu[s], n = st.page[s];
    st.cu[s] = static_cast<int32_t>(a);
    st.page[s] = static_cast<int32_t>(b);
    a += q;
    b += n;
  }
  if (threadIdx.x == 0) {
    st.cu[S] = static_cast<int32_t>(ta);
    st.page[S] = static_cast<int32_t>(tb);
  }
  __syncthreads();
}

// Entry j of segment s's table row: a held page, a new page (also entered
// into the request's own row), or -1.
__device__ __forceinline__ int32_t table_entry(const StepArgs& p, const int32_t* row, int32_t j,
                                               int32_t held, int32_t after, const int32_t* fresh) {
  if (j < held) return row[j];
  return j < after ? fresh[j - held] : -1;
}

__global__ void __launch_bounds__(kThreads) build_tables_kernel(const StepArgs p) {
  extern __shared__ char smem[];
  Step st;
  load_step<false>(p, st, smem);
  const int32_t S = p.S, lg = p.P_log2, width = p.width;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0 && st.bad && p.err) atomicOr(p.err, st.bad);
    for (int s = threadIdx.x; s <= S; s += kThreads) {
      p.cu[s] = st.cu[s];
      if (s < S) p.sk[s] = st.have[s] + st.cu[s + 1] - st.cu[s];
    }
    if (p.rows) {
      // the last token of every segment that has one, in segment order
      const int per = (S + kThreads - 1) / kThreads;
      const int s0 = min(S, static_cast<int>(threadIdx.x) * per), s1 = min(S, s0 + per);
      int64_t n = 0, none = 0, total, t2;
      for (int s = s0; s < s1; ++s) n += st.cu[s + 1] > st.cu[s];
      block_scan2(n, none, total, t2);
      for (int s = s0; s < s1; ++s)
        if (st.cu[s + 1] > st.cu[s]) p.rows[n++] = st.cu[s + 1] - 1;
      for (int s = static_cast<int>(total) + threadIdx.x; s < S; s += kThreads) p.rows[s] = -1;
    }
  }
  const int32_t per_row = (width + kPiece - 1) / kPiece;
  const int64_t table_pieces = static_cast<int64_t>(S) * per_row;
  const int64_t pieces = table_pieces + (p.max_tokens + kPiece - 1) / kPiece;
  const bool vec = (width & 3) == 0;  // rows 16-byte aligned
  for (int64_t w = blockIdx.x; w < pieces; w += gridDim.x) {
    if (w < table_pieces) {
      const int32_t s = static_cast<int32_t>(w / per_row);
      const int32_t j0 = static_cast<int32_t>(w - static_cast<int64_t>(s) * per_row) * kPiece;
      const int32_t j1 = min(width, j0 + kPiece);
      const int32_t id = st.id[s];
      const int32_t held = pages_of(st.have[s], lg);
      const int32_t after = pages_of(st.have[s] + st.cu[s + 1] - st.cu[s], lg);
      int32_t* row = p.request_pages + static_cast<int64_t>(id < 0 ? 0 : id) * width;
      const int32_t* fresh = p.free_pages + st.base + st.page[s];
      int32_t* dst = p.bt + static_cast<int64_t>(s) * width;
      if (vec) {
        for (int32_t j = j0 + 4 * threadIdx.x; j < j1; j += 4 * kThreads) {
          int4 v;
          if (j + 4 <= held) {
            v = *reinterpret_cast<const int4*>(row + j);
          } else if (j >= after) {
            v = make_int4(-1, -1, -1, -1);
          } else {
            v.x = table_entry(p, row, j, held, after, fresh);
            v.y = table_entry(p, row, j + 1, held, after, fresh);
            v.z = table_entry(p, row, j + 2, held, after, fresh);
            v.w = table_entry(p, row, j + 3, held, after, fresh);
          }
          *reinterpret_cast<int4*>(dst + j) = v;
        }
      } else {
        for (int32_t j = j0 + threadIdx.x; j < j1; j += kThreads)
          dst[j] = table_entry(p, row, j, held, after, fresh);
      }
      // new pages go behind the held ones (nothing else reads or writes there)
      for (int32_t j = max(j0, held) + threadIdx.x; j < min(j1, after); j += kThreads)
        row[j] = fresh[j - held];
    } else {
      const int32_t t0 = static_cast<int32_t>(w - table_pieces) * kPiece;
      const int32_t t1 = min(p.max_tokens, t0 + kPiece), T = st.cu[S];
      for (int32_t t = t0 + threadIdx.x; t < t1; t += kThreads) {
        int64_t slot = -1;
        int32_t at = 0;
        if (t < T) {
          int lo = 0, hi = S;  // the last segment that begins at or before t and is not empty
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (st.cu[mid] <= t) lo = mid;
            else hi = mid;
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
// lengths and the count move on.  `finish`: the launch's one CTA (or the
// second launch's) writes lengths and count once every page was read; the
// copies touch only free_pages, so both launches read the same state.
__global__ void __launch_bounds__(kThreads)
    commit_kernel(const StepArgs p, const bool copy, const bool finish) {
  extern __shared__ char smem[];
  Step st;
  load_step<true>(p, st, smem);
  const int32_t S = p.S, lg = p.P_log2, width = p.width;
  if (finish && threadIdx.x == 0 && st.bad && p.err) atomicOr(p.err, st.bad);
  if (st.bad) return;
  if (copy) {
    const int32_t per_row = (width + kPiece - 1) / kPiece;
    const int64_t pieces = static_cast<int64_t>(S) * per_row;
    for (int64_t w = blockIdx.x; w < pieces; w += gridDim.x) {
      const int32_t s = static_cast<int32_t>(w / per_row);
      if (st.id[s] < 0) continue;
      const int32_t after = pages_of(st.have[s] + st.cu[s + 1] - st.cu[s], lg);
      const int32_t keep = after - (st.page[s + 1] - st.page[s]);
      const int32_t j0 = static_cast<int32_t>(w - static_cast<int64_t>(s) * per_row) * kPiece;
      const int32_t* row = p.request_pages + static_cast<int64_t>(st.id[s]) * width;
      int32_t* to = p.free_pages + st.base + st.page[s] - keep;
      for (int32_t j = max(j0, keep) + threadIdx.x; j < min(j0 + kPiece, after); j += kThreads)
        to[j] = row[j];
    }
  }
  if (finish) {
    __syncthreads();
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

// CTAs for `entries` words of work: one per piece, at most two per SM (each
// repeats the prefix sums).
int grid_of(int64_t pieces) {
  const int64_t cap = 2 * static_cast<int64_t>(step_num_sms());
  return static_cast<int>(pieces < 1 ? 1 : pieces > cap ? cap : pieces);
}

}  // namespace

int step_num_sms() {
  static thread_local int dev_of = -1, sms = 148;
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
  const size_t smem = step_smem(num_seqs, a.R);
  if (const int e = allow_smem<build_tables_kernel>(static_cast<int>(step_smem(kMaxStepSeqs, kWindow)))) return e;
  const int64_t pieces =
      static_cast<int64_t>(num_seqs) * ((a.width + kPiece - 1) / kPiece) +
      (static_cast<int64_t>(max_tokens) + kPiece - 1) / kPiece;
  build_tables_kernel<<<grid_of(pieces), kThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return static_cast<int>(cudaGetLastError());
}

int launch_commit_step(const mcp_request_pool& pool, const int32_t* request_ids,
                       const int32_t* q_lens, const int32_t* new_lens, int32_t num_seqs,
                       int32_t* error_word, void* stream) {
  StepArgs a = step_args(pool, request_ids, q_lens, num_seqs, error_word);
  a.new_lens = new_lens;
  const size_t smem = step_smem(num_seqs, a.R);
  if (const int e = allow_smem<commit_kernel>(static_cast<int>(step_smem(kMaxStepSeqs, kWindow)))) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t pieces = static_cast<int64_t>(num_seqs) * ((a.width + kPiece - 1) / kPiece);
  // a commit that keeps every token returns no page: one CTA moves the lengths on
  const int grid = new_lens ? grid_of(pieces) : 1;
  if (grid <= 16) {
    commit_kernel<<<1, kThreads, smem, st>>>(a, new_lens != nullptr, true);
  } else {
    commit_kernel<<<grid, kThreads, smem, st>>>(a, true, false);
    commit_kernel<<<1, kThreads, smem, st>>>(a, false, true);
  }
  return static_cast<int>(cudaGetLastError());
}

}  // namespace mcp
