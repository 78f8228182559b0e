// Trees of drafted tokens: which tokens of its tree each token sees, and the
// move of an accepted path's K/V to the front of its segment.
//
// A tree's token i has a parent before it (or none); it sees
//   seen(i) = seen(parent) and i,   at position history + |seen(i)| - 1.
#include <cuda_runtime.h>
#include <stdint.h>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

// ------------------------------------------------------------------- masks
struct MaskArgs {
  const int32_t* parents;
  const int32_t* cu;
  const int32_t* sk;
  const int32_t* mask_rows;
  uint32_t* mask;
  int32_t* positions;
  int32_t* err;
  int32_t T, rows, W;
  int32_t lanes_log2;  // threads of a token: W rounded up to a power of two
};

// A CTA a segment.  The rows are filled by doubling: row[i] holds the tokens
// from i up to, but without, up[i]; each round takes over row[up[i]] and
// up[up[i]], so a tree of depth d takes log2(d) rounds where a walk up takes d
// steps.  A row that another thread has already extended in the same round only
// holds more of the same ancestors; up, which must not run ahead of the rows, is
// written to a second array.  Depth is the number of bits.
//
// Bound by its launch and the chain of loads in front of the rounds (1024 trees of 48
// to 128 tokens 6.5 us, 4 of 16 2.9); with 256 threads 8 trees of 1024 tokens took 54.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) tree_masks_kernel(const MaskArgs p) {
  extern __shared__ uint32_t smem[];
  const int s = blockIdx.x, tid = threadIdx.x, W = p.W;
  const int t0 = p.cu[s], t1 = p.cu[s + 1];
  if (t1 <= t0) {  // compared as they are: the difference of wild bounds leaves 32 bits
    if (t1 < t0 && tid == 0 && p.err) atomicOr(p.err, MCP_DEVERR_SEGMENT);
    return;
  }
  const int n = static_cast<int>(min(static_cast<int64_t>(t1) - t0, static_cast<int64_t>(0x7fffffff)));
  const int hist = p.sk[s] - n, m0 = p.mask_rows[s];
  int bad = p.sk[s] < n ? MCP_DEVERR_SEGMENT : 0;
  const bool outside = t0 < 0 || t1 > p.T;
  if (outside) bad |= MCP_DEVERR_SEGMENT;
  const bool tree = m0 >= 0;
  const bool large = tree && (n > 32 * W || m0 > p.rows - n);
  if (large) bad |= MCP_DEVERR_TREE;
  if (bad && tid == 0 && p.err) atomicOr(p.err, bad);
  if (outside || large) return;
  if (!tree) {
    if (p.positions)
      for (int i = tid; i < n; i += kThreads) p.positions[t0 + i] = hist + i;
    return;
  }
  uint32_t* row = smem;                                         // [n][W]
  int32_t* up = reinterpret_cast<int32_t*>(smem + 32 * W * W);  // two of [32 W]
  int32_t* next = up + 32 * W;
  // a thread takes word `w` of tokens i0, i0 + step, ..; words behind a token's own
  // stay 0
  const int w = tid & ((1 << p.lanes_log2) - 1), i0 = tid >> p.lanes_log2, step = kThreads >> p.lanes_log2;
  bool some = false;
  for (int i = tid; i < n; i += kThreads) {
    int32_t a = p.parents[t0 + i];
    if (a >= i) {
      if (p.err) atomicOr(p.err, MCP_DEVERR_TREE);
      a = -1;
    }
    up[i] = a < 0 ? -1 : a;
    some |= a >= 0;
  }
  if (w < W)
    for (int i = i0; i < n; i += step) row[i * W + w] = w == i >> 5 ? 1u << (i & 31) : 0u;
  while (__syncthreads_or(some)) {
    some = false;
#pragma unroll 4
    for (int i = i0; i < n; i += step) {
      const int a = up[i];
      if (a >= 0 && w <= a >> 5) row[i * W + w] |= row[a * W + w];
    }
    for (int i = tid; i < n; i += kThreads) {
      const int a = up[i];
      const int b = a >= 0 ? up[a] : -1;
      next[i] = b;
      some |= b >= 0;
    }
    int32_t* const t = up;
    up = next;
    next = t;
  }
  uint32_t* out = p.mask + static_cast<int64_t>(m0) * W;
  for (int x = tid; x < n * W; x += kThreads) out[x] = row[x];
  if (p.positions)
    for (int base = 0; base < n; base += step) {  // the words of a token lie in its threads' lanes
      const int i = base + i0;
      int bits = w < W && i < n ? __popc(row[i * W + w]) : 0;
      for (int o = 1 << p.lanes_log2 >> 1; o > 0; o >>= 1) bits += __shfl_xor_sync(0xffffffffu, bits, o);
      if (w == 0 && i < n) p.positions[t0 + i] = hist + bits - 1;
    }
}

// -------------------------------------------------------------------- keep
constexpr int kKeepThreads = 256;
constexpr int kKeepLayers = 64;  // whose addresses fit a launch's arguments
constexpr int kKeepSlots = 256;  // moves whose slots a CTA has at hand
constexpr int kKeepBatch = 8;    // rows in flight a thread

// K and V of each layer: listed, or all layers' at one distance
struct ListedCaches {
  uint4* at[2 * kKeepLayers];
  __device__ __forceinline__ uint4* operator[](int i) const { return at[i]; }
};
struct EvenCaches {
  uint4* at[2];
  int64_t stride;  // in 16 bytes
  __device__ __forceinline__ uint4* operator[](int i) const { return at[i & 1] + (i >> 1) * stride; }
};
struct KeepArgs {
  const int32_t* bt;
  const int32_t* cu;
  const int32_t* sk;
  const int32_t* cu_rows;
  const int32_t* accepted;
  const int32_t* path;
  int32_t* new_lens;
  int32_t* err;
  int32_t total_rows, page_log2, max_pages, num_pages, vec;
  int32_t columns;   // 16-byte columns of all layers' K and V rows: 2 * layers * vec
  int32_t per_cta;   // columns of a CTA, a multiple of its threads
  int32_t chunks;    // CTAs of a segment
};

// Slot of position `pos`, -1 (and an error bit) where its page is none of the pool's
__device__ __forceinline__ int64_t slot_of(const KeepArgs& p, const int32_t* bt, int pos, int& bad) {
  const int32_t page = bt[pos >> p.page_log2];
  if (page < 0 || page >= p.num_pages) {
    bad |= MCP_DEVERR_PAGE_RANGE;
    return -1;
  }
  return (static_cast<int64_t>(page) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
}

// A CTA moves some 16-byte columns of the rows of all layers for one segment.
// One thread takes a column through all moves in their order, up to kKeepBatch of
// them loaded before the first is stored: a path rises strictly, so move k reads
// place path[k] >= k, which only moves after it write.
//
// Bound by HBM behind the chain lengths -> path -> pages -> rows: 64 paths in 32 layers
// (25 MB each way) 12.4 us, 4 TB/s with the launch; one path 2.7 us, its launch.  Four
// rows in flight a thread and twice the threads 12.0, a CTA of 128 threads 12.4.
template <typename Caches>
__global__ void __launch_bounds__(kKeepThreads)
    keep_path_kernel(const __grid_constant__ KeepArgs p, const __grid_constant__ Caches caches) {
  __shared__ int64_t from[kKeepSlots], to[kKeepSlots];
  const int s = blockIdx.x / p.chunks, chunk = blockIdx.x - s * p.chunks, tid = threadIdx.x;
  const int sk = p.sk[s], r0 = p.cu_rows[s], r1 = p.cu_rows[s + 1], m = p.accepted[s];
  const int64_t tokens = static_cast<int64_t>(p.cu[s + 1]) - p.cu[s];
  const int lq = static_cast<int>(tokens), hist = sk - lq, n = r1 - r0;  // used of sound segments only
  int bad = 0;
  bool move = n == lq && lq > 0;
  if (tokens < 0 || sk < tokens || r1 < r0 || r0 < 0 || r1 > p.total_rows ||
      sk > static_cast<int64_t>(p.max_pages) << p.page_log2) {
    bad = MCP_DEVERR_SEGMENT;
    move = false;
  } else if (move && (m < 0 || m > n)) {
    bad = MCP_DEVERR_TREE;
    move = false;
  }
  if (move) {  // the whole path before the first move
    bool sound = true;
    for (int k = tid; k < m; k += kKeepThreads) {
      const int a = p.path[r0 + k], before = k ? p.path[r0 + k - 1] : -1;
      sound &= a > before && a < n && a >= 0;
    }
    if (!__syncthreads_and(sound)) {
      bad = MCP_DEVERR_TREE;
      move = false;
    }
  }
  if (chunk == 0 && tid == 0) {
    if (p.new_lens) p.new_lens[s] = move ? hist + m : sk;
    if (bad && p.err) atomicOr(p.err, bad);
  }
  if (!move) return;
  const int32_t* bt = p.bt + static_cast<int64_t>(s) * p.max_pages;
  const int c0 = chunk * p.per_cta, c1 = min(c0 + p.per_cta, p.columns);
  for (int k0 = 0; k0 < m; k0 += kKeepSlots) {
    const int left = min(kKeepSlots, m - k0);
    if (tid < left) {
      const int a = p.path[r0 + k0 + tid], k = k0 + tid;
      int64_t src = -1, dst = -1;
      if (a != k) {
        int page_bad = 0;
        src = slot_of(p, bt, hist + a, page_bad);
        dst = slot_of(p, bt, hist + k, page_bad);
        if (page_bad) {
          src = -1;
          if (chunk == 0 && p.err) atomicOr(p.err, page_bad);
        }
      }
      from[tid] = src;
      to[tid] = dst;
    }
    __syncthreads();
    for (int c = c0 + tid; c < c1; c += kKeepThreads) {
      const int which = c / p.vec;
      uint4* cache = caches[which] + (c - which * p.vec);
      for (int b = 0; b < left; b += kKeepBatch) {
        uint4 v[kKeepBatch];
#pragma unroll
        for (int j = 0; j < kKeepBatch; ++j)
          if (b + j < left && from[b + j] >= 0) v[j] = cache[from[b + j] * p.vec];
#pragma unroll
        for (int j = 0; j < kKeepBatch; ++j)
          if (b + j < left && from[b + j] >= 0) cache[to[b + j] * p.vec] = v[j];
      }
    }
    __syncthreads();
  }
}

}  // namespace

int launch_build_tree_masks(const int32_t* parents, const int32_t* cu_seqlens_q,
                            const int32_t* seqlens_k, const int32_t* mask_rows, int32_t num_seqs,
                            int32_t total_tokens, int32_t num_mask_rows, int32_t mask_words,
                            int32_t* tree_mask, int32_t* positions, int32_t* error_word,
                            void* stream) {
  const int smem = 4 * (32 * mask_words * mask_words + 2 * 32 * mask_words);  // at most 136 KB
  MaskArgs a = {parents, cu_seqlens_q, seqlens_k, mask_rows, reinterpret_cast<uint32_t*>(tree_mask),
                positions, error_word, total_tokens, num_mask_rows, mask_words, 0};
  while (1 << a.lanes_log2 < mask_words) ++a.lanes_log2;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (mask_words <= 4) {  // up to 128 tokens: two words a thread
    tree_masks_kernel<256><<<num_seqs, 256, smem, st>>>(a);
  } else {
    const int e = allow_smem<tree_masks_kernel<1024>>(4 * (32 * 32 * 32 + 2 * 32 * 32));
    if (e != 0) return e;
    tree_masks_kernel<1024><<<num_seqs, 1024, smem, st>>>(a);
  }
  return static_cast<int>(cudaGetLastError());
}

int launch_kv_keep_path(const mcp_keep_desc& d, void* const* k_caches, void* const* v_caches,
                        const int32_t* block_tables, const int32_t* cu_seqlens_q,
                        const int32_t* seqlens_k, const int32_t* cu_rows, const int32_t* accepted,
                        const int32_t* path, int32_t* new_lens, int32_t* error_word, void* stream) {
  KeepArgs a;
  a.bt = block_tables;
  a.cu = cu_seqlens_q;
  a.sk = seqlens_k;
  a.cu_rows = cu_rows ? cu_rows : cu_seqlens_q;
  a.accepted = accepted;
  a.path = path;
  a.new_lens = new_lens;
  a.err = error_word;
  a.total_rows = d.total_rows;
  a.page_log2 = __builtin_ctz(static_cast<unsigned>(d.page_size));
  a.max_pages = d.max_pages_per_seq;
  a.num_pages = d.num_pages;
  a.vec = static_cast<int32_t>(static_cast<int64_t>(d.num_kv_heads) * d.head_dim / 8);
  auto launch = [&](const auto& caches, int layers) {
    a.columns = 2 * layers * a.vec;
    // a column a thread, more of them where that would be over the 4 CTAs an SM that
    // its registers hold (64 paths in 32 layers: 12.4 us; 8 CTAs 13.0, 16 14.8)
    const int64_t all = static_cast<int64_t>(d.num_seqs) * ((a.columns + kKeepThreads - 1) / kKeepThreads);
    const int64_t rounds = (all + 4LL * step_num_sms() - 1) / (4LL * step_num_sms());
    const int64_t per = kKeepThreads * (rounds < 1 ? 1 : rounds);
    a.per_cta = static_cast<int32_t>(per < a.columns ? per : (a.columns > 0 ? a.columns : 1));
    a.chunks = a.columns > 0 ? (a.columns + a.per_cta - 1) / a.per_cta : 1;
    const int64_t grid = static_cast<int64_t>(d.num_seqs) * a.chunks;
    keep_path_kernel<<<static_cast<unsigned>(grid), kKeepThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, caches);
    return static_cast<int>(cudaGetLastError());
  };
  if (d.layer_stride != 0 && d.num_layers > 0) {  // without layers there is no address to read
    const EvenCaches caches = {{static_cast<uint4*>(k_caches[0]), static_cast<uint4*>(v_caches[0])},
                               d.layer_stride / 8};
    return launch(caches, d.num_layers);
  }
  for (int l0 = 0; l0 == 0 || l0 < d.num_layers; l0 += kKeepLayers) {
    const int layers = d.num_layers - l0 < kKeepLayers ? d.num_layers - l0 : kKeepLayers;
    ListedCaches caches = {};
    for (int l = 0; l < layers; ++l) {
      caches.at[2 * l] = static_cast<uint4*>(k_caches[l0 + l]);
      caches.at[2 * l + 1] = static_cast<uint4*>(v_caches[l0 + l]);
    }
    const int e = launch(caches, layers);
    if (e != 0) return e;
  }
  return 0;
}

}  // namespace mcp
