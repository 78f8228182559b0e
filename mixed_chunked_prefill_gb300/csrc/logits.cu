// What the sampled rows' logits go through between the output head and the
// sampler: which tokens each request has had, kept on the GPU, and biases,
// penalties for repeated tokens, temperature and grammar masks.
//
// [W] "采样：只有该出字的请求才出字": logits exist only for the rows at
// logits_indices; each row belongs to a request, and a request's state here is
//   seen   [2][W] words: bit v of plane 0 = token v is in the prompt, of plane
//          1 = it was sampled (W = ceil(vocab / 32))
//   counts [32 W]: how often token v was sampled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

// ------------------------------------------------------------- token counts
constexpr int kCountThreads = 256;

struct CountArgs {
  const int32_t* ids;
  const int32_t* tokens;
  const int32_t* cu;  // NULL: token i belongs to row i
  int32_t* seen;
  int32_t* counts;
  int32_t* err;
  int32_t rows, n, R, V, W, prompt;
};

// Clear the rows' state: both planes whole, counts only where a bit says that
// one may be there (a row of counts is 32 times its plane).
__global__ void __launch_bounds__(kCountThreads) clear_counts_kernel(const CountArgs p) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t total = static_cast<int64_t>(p.rows) * p.W;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCountThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kCountThreads) {
    const int32_t r = static_cast<int32_t>(i / p.W), w = static_cast<int32_t>(i - static_cast<int64_t>(r) * p.W);
    const int32_t id = p.ids[r];
    if (id >= p.R && w == 0 && p.err) atomicOr(p.err, MCP_DEVERR_REQUEST);
    if (id < 0 || id >= p.R) continue;
    int32_t* seen = p.seen + static_cast<int64_t>(id) * 2 * p.W + w;
    uint32_t had = static_cast<uint32_t>(seen[p.W]);
    seen[0] = 0;
    seen[p.W] = 0;
    int32_t* c = p.counts + (static_cast<int64_t>(id) * p.W + w) * 32;
    while (had) {
      c[__ffs(had) - 1] = 0;
      had &= had - 1;
    }
  }
}

// First row that ends behind token c (`rows`: none), looked up by all threads of
// the CTA together: their loads are in flight at once, where a binary search
// makes one after the other.
template <int kThreads>
__device__ __forceinline__ int32_t first_row(const CountArgs& p, int32_t c) {
  int32_t n = 0;
  for (int32_t s0 = 0; s0 < p.rows; s0 += kThreads) {
    const int32_t s = s0 + threadIdx.x;
    const int32_t here = __syncthreads_count(s < p.rows && p.cu[s + 1] <= c);
    n += here;
    if (here < kThreads) break;
  }
  return n;
}
// The row that token i is in, not before `lo` (-1: in none)
__device__ __forceinline__ int32_t row_of(const CountArgs& p, int32_t i, int32_t lo) {
  if (lo < p.rows && p.cu[lo + 1] <= i) {
    ++lo;
    if (lo < p.rows && p.cu[lo + 1] <= i) {
      int32_t hi = p.rows;
      while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (p.cu[mid + 1] <= i) lo = mid + 1;
        else hi = mid;
      }
    }
  }
  return lo < p.rows && p.cu[lo] <= i ? lo : -1;
}

// A token of row `row` (-1: of none), added where it belongs.  Adding and marking
// are atomic, so the result does not depend on the order and a request may stand
// in several rows; a mark that is already there is only read (text repeats few
// words very often).  Returns error bits.
__device__ __forceinline__ int add_token(const CountArgs& p, int32_t tok, int32_t row) {
  const int32_t id = row < 0 ? -1 : p.ids[row];
  if (id < 0 || tok < 0) return id >= p.R ? MCP_DEVERR_REQUEST : 0;
  if (id >= p.R) return MCP_DEVERR_REQUEST;
  if (tok >= p.V) return MCP_DEVERR_TOKEN_RANGE;
  int32_t* word = p.seen + (static_cast<int64_t>(id) * 2 + (p.prompt ? 0 : 1)) * p.W + (tok >> 5);
  const uint32_t had = *reinterpret_cast<volatile uint32_t*>(word), bit = 1u << (tok & 31);
  if (!p.prompt) atomicAdd(p.counts + static_cast<int64_t>(id) * 32 * p.W + tok, 1);
  if (!(had & bit)) atomicOr(reinterpret_cast<unsigned int*>(word), bit);
  return 0;
}

// A thread a token: the chain of loads from the row's end to the mark is what
// this takes (250 sampled tokens 3.0 us, 2.3 of them the launch).
__global__ void __launch_bounds__(kCountThreads) add_tokens_kernel(const CountArgs p) {
  const int32_t c = blockIdx.x * kCountThreads, i = c + threadIdx.x;
  const int32_t tok = i < p.n ? p.tokens[i] : -1;
  int32_t row = i;
  if (p.cu) row = row_of(p, i, first_row<kCountThreads>(p, c));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows are cleared
  if (i >= p.n) return;
  const int bad = add_token(p, tok, row);
  if (bad && p.err) atomicOr(p.err, bad);
}

// Long texts.  A CTA takes `chunk` tokens and marks those of one row in a bitmap
// in shared memory, whose words then go to the row by one atomic each, 32
// neighbouring ones a warp: a cleared row whose most frequent tokens were marked
// one by one took hundreds of atomics on the same word.  The bitmap is filled
// while the launch before clears the rows.  Parts of rows shorter than kDense
// tokens are not worth a pass over it.
//
// Taken from 4096 tokens and an average of 2048 a row on.  Prompts marked like
// this and token by token, rows cleared first, us: 64 of 500 tokens 8.6 / 6.1,
// 64 of 4000 8.5 / 9.1, 64 of 8000 8.6 / 13.6, 64 of 32768 11.7 / 38.  Sampled
// tokens have their counts' atomics beside the marks: from 8192 a row on (64 of
// 4096 6.4 / 5.0, 64 of 32768 22 / 33).
constexpr int kMarkThreads = 1024;
constexpr int kDense = 1024;
constexpr int kMarkTokens = 4096, kMarkRow = 2048, kCountRow = 8192;
constexpr int kMapTokens = 1 << 18;  // 32 KB; tokens from there on are marked one by one

__global__ void __launch_bounds__(kMarkThreads) mark_texts_kernel(const CountArgs p, const int32_t chunk) {
  extern __shared__ __align__(16) uint32_t map[];
  const int32_t mapped = min(p.V, kMapTokens), words = (mapped + 31) / 32;
  for (int w = threadIdx.x; w < words; w += kMarkThreads) map[w] = 0;
  const bool vec = (reinterpret_cast<uintptr_t>(p.tokens) & 15) == 0;
  int32_t c = blockIdx.x * chunk;
  const int32_t c1 = min(p.n, c + chunk);
  int bad = 0;
  int32_t row = first_row<kMarkThreads>(p, c);
  if (!p.prompt) asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();  // the cleared map
  while (c < c1 && row < p.rows) {
    const int32_t begin = p.cu[row], end = min(c1, p.cu[row + 1]);
    if (end <= c) {  // rows without tokens
      row = max(row + 1, first_row<kMarkThreads>(p, c));
      continue;
    }
    if (begin > c) {  // tokens before the first row
      c = min(c1, begin);
      continue;
    }
    if (end - c < kDense) {
      const int32_t i = c + threadIdx.x;
      const int32_t r = i < c1 ? row_of(p, i, row) : -1;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (r >= 0) bad |= add_token(p, p.tokens[i], r);
      c = min(c1, c + kMarkThreads);
      row = end < c ? first_row<kMarkThreads>(p, c) : row;
      continue;
    }
    const int32_t id = p.ids[row];
    if (id >= p.R) bad |= MCP_DEVERR_REQUEST;
    if (id >= 0 && id < p.R) {
      uint32_t* seen = reinterpret_cast<uint32_t*>(p.seen) + (static_cast<int64_t>(id) * 2 + (p.prompt ? 0 : 1)) * p.W;
      int32_t* counts = p.counts + static_cast<int64_t>(id) * 32 * p.W;
      auto mark = [&](int32_t tok) {
        if (tok < 0) return;
        if (tok >= p.V) {
          bad |= MCP_DEVERR_TOKEN_RANGE;
          return;
        }
        if (!p.prompt) atomicAdd(counts + tok, 1);
        const uint32_t bit = 1u << (tok & 31);
        if (tok < mapped) {
          if (!(map[tok >> 5] & bit)) atomicOr(map + (tok >> 5), bit);
        } else {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          atomicOr(seen + (tok >> 5), bit);
        }
      };
      if (vec) {  // whole vectors of four tokens, those that reach into a neighbour token by token
        const int32_t a0 = (c + 3) & ~3, a1 = end & ~3;
        if (threadIdx.x < a0 - c) mark(p.tokens[c + threadIdx.x]);
        if (threadIdx.x < end - a1) mark(p.tokens[a1 + threadIdx.x]);
#pragma unroll 2
        for (int32_t i = a0 + 4 * static_cast<int32_t>(threadIdx.x); i < a1; i += 4 * kMarkThreads) {
          const int4 q = *reinterpret_cast<const int4*>(p.tokens + i);
          mark(q.x), mark(q.y), mark(q.z), mark(q.w);
        }
      } else {
#pragma unroll 4
        for (int32_t i = c + static_cast<int32_t>(threadIdx.x); i < end; i += kMarkThreads) mark(p.tokens[i]);
      }
      __syncthreads();
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int w = threadIdx.x; w < words; w += kMarkThreads) {
        const uint32_t v = map[w];
        if (v) {
          atomicOr(seen + w, v);
          map[w] = 0;
        }
      }
      __syncthreads();
    }
    c = end;
    ++row;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows this launch follows the clearing too
  if (bad && p.err) atomicOr(p.err, bad);
}

// ------------------------------------------------------------------- logits
// Per row, for every token v, in fp32 and rounded once:
//   x += bias[v];  x = x > 0 ? x / rho : x rho   where v was seen
//   x -= frequency count[v] + presence           where count[v] > 0
//   x /= temperature (if > 0);  x = -inf         where the mask's bit is 0
//
// One pass.  What has to move is the logits, three bits a token and the counts
// of the tokens that were sampled (each 8 tokens' counts are one 32-byte
// sector, read only where plane 1 has a bit).  In place and without a
// temperature nothing but seen, biased and masked tokens changes, so nothing
// else is read or written.  A masked token's logit and count are not read.
struct LogitArgs {
  const void* logits;
  void* out;
  const int32_t* ids;
  const int32_t* seen;
  const int32_t* counts;
  const float* temperature;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_offsets;
  const int32_t* bias_tokens;
  const float* bias_values;
  const int32_t* mask;
  const int32_t* mask_rows;
  int32_t* err;
  int64_t ld_in, ld_out;
  int32_t rows, V, W, R, num_bias, num_masks, inplace;
  int32_t tiles, parts;  // tiles of a CTA, CTAs of a row
};

constexpr int kLogitThreads = 256;
constexpr int kLogitTile = 16 * kLogitThreads;  // tokens of one row that a CTA takes at a time
constexpr int kLogitMaxTiles = 4;               // tiles of one CTA
constexpr int kLogitSlots = 2;                  // tiles of logits in flight

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

template <typename T, int n>
struct alignas(n * sizeof(T)) Vec {
  T v[n];
};

// 1 / t for products: hi the part that fp32 holds, cut off, and lo > 0 what is left
// of it, so that x / t = x hi + x lo is off by its one rounding (and 2^-46), and of an
// infinite x both are infinite alike.  t from 2^-123 to 2^64.
struct Reciprocal {
  float hi, lo;
  __device__ __forceinline__ explicit Reciprocal(float t) {
    hi = __frcp_rz(t);
    lo = fmaxf(hi * fmaf(-t, hi, 1.f), hi * 0x1p-60f);
  }
  __device__ __forceinline__ float times(float x) const { return fmaf(x, hi, x * lo); }
};

// The bias of token `tok`, which has one: entries [lo, hi) in rising order.
template <typename Tokens, typename Values>
__device__ __forceinline__ float find_bias(Tokens tokens, Values values, int32_t lo, int32_t hi, int32_t tok) {
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (tokens[mid] <= tok) lo = mid;
    else hi = mid;
  }
  return tokens[lo] == tok ? values[lo] : 0.f;
}

// 4, 8 or 16 bytes global -> shared without a register in between
template <int n>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// kWhole, kShifted: a thread takes 4 neighbouring tokens at a time, 8 bytes of
// 16-bit logits in and 16 bytes of fp32 out.  A row that starts between those
// addresses (an odd vocabulary: kShifted) is taken from up to 3 tokens before
// its start, so that the accesses are aligned; its groups' bits then come from
// two words.  kSingle, a warp on 32 neighbouring tokens: logits and out whose
// rows are aligned differently.
//
// What bounds the pass is how many bytes are in flight.  A CTA reads all bits
// of its part into shared memory at once, so that it knows which logits it
// needs, and a ring of tiles in shared memory takes those (asynchronous
// copies: no registers, and a thread reads only what it copied itself).
//
// Most tokens were neither seen nor biased: the pass gives them a conversion, a
// product with 1 / temperature and a select, and leaves the others out.  Those
// are listed and taken afterwards, one a thread (a row's first biases are kept
// in shared memory for that: looked up in global memory, 16 biases a row took 15
// us longer for 512 rows).
//
// 512 rows of 128000 tokens, bf16 to fp32, us: 65 without anything seen (6.3
// TB/s), 74 with 2000 seen tokens a row; half of the rows masked, 64 and 71.
// Beside the traffic it is the phases of a CTA, each of which begins with loads
// that nothing hides but the SM's other CTAs.
enum LogitRows { kWhole, kShifted, kSingle };

constexpr int kLogitPlanes = 5;  // changed, sampled, allowed, biased, seen (prompt or sampled)
constexpr int kLogitWords = kLogitMaxTiles * kLogitTile / 32;  // of a plane, in a part
// CTAs of an SM: tiles in flight beyond two, or longer parts, are worth less than
// more CTAs (512 rows of 128000, us: 6 CTAs of 4 tiles 74, of 2 77, of 6 82; 5 CTAs
// with three in flight 75; 4 CTAs of 8 tiles with four in flight 83).
template <typename T>
constexpr int kLogitCtas = sizeof(T) == 2 ? 6 : 4;
template <typename T>
constexpr int kLogitRing = kLogitSlots * kLogitTile * static_cast<int>(sizeof(T));
template <typename T>
constexpr int kLogitSmem = kLogitPlanes * 4 * (kLogitWords + 2) + kLogitRing<T>;

template <typename TI, typename TO, int kRows>
__global__ void __launch_bounds__(kLogitThreads, kLogitCtas<TI>) process_logits_kernel(const LogitArgs p) {
  constexpr int kVec = kRows == kSingle ? 1 : 4;
  constexpr int kGroups = kLogitTile / kLogitThreads / kVec;  // of a thread and tile
  constexpr uint32_t kAll = (1u << kVec) - 1;
  constexpr bool kAsync = kVec * sizeof(TI) >= 4;
  constexpr int kSlots = kLogitSlots;
  extern __shared__ __align__(16) unsigned char lsmem[];
  TI* ring = reinterpret_cast<TI*>(lsmem);
  uint32_t* plane = reinterpret_cast<uint32_t*>(lsmem + kLogitRing<TI>);
  __shared__ int32_t s_tok[kLogitThreads];  // the row's first biases
  __shared__ float s_val[kLogitThreads];
  __shared__ int32_t s_total, s_listed;  // tokens of plane 0, of the list
  constexpr int kPlane = kLogitWords + 2;

  const int32_t row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
  const int32_t id = p.ids ? p.ids[row] : 0;
  const int32_t mrow = !p.mask ? -1 : p.mask_rows ? p.mask_rows[row] : row;
  int32_t lo = 0, hi = 0;  // the row's biases
  if (p.bias_offsets) lo = p.bias_offsets[row], hi = p.bias_offsets[row + 1];
  if (id < 0) return;  // padding: the row stays as it was
  if ((p.ids && id >= p.R) || mrow >= p.num_masks) {
    if (part == 0 && threadIdx.x == 0 && p.err) atomicOr(p.err, MCP_DEVERR_REQUEST);
    return;
  }
  // tokens of this CTA: [begin, end), those below 0 do not exist
  const int32_t shift =
      kRows != kShifted ? 0 : static_cast<int32_t>((reinterpret_cast<uintptr_t>(p.out) / sizeof(TO) + row * p.ld_out) % 4);
  const int32_t begin = part * p.tiles * kLogitTile - shift;
  const int32_t end = min(p.V, begin + p.tiles * kLogitTile);
  if (begin >= end) return;
  const int32_t word0 = begin >> 5;  // of the planes' first entry (-1: one word of zeros)
  const int32_t nwords = ((end - 1) >> 5) - word0 + 1;
  const uint32_t* seen =
      p.ids ? reinterpret_cast<const uint32_t*>(p.seen) + static_cast<int64_t>(id) * 2 * p.W : nullptr;
  const uint32_t* mask =
      mrow < 0 ? nullptr : reinterpret_cast<const uint32_t*>(p.mask) + static_cast<int64_t>(mrow) * p.W;
  int bad = 0;
  if (lo < 0 || hi < lo || hi > p.num_bias) {
    bad = MCP_DEVERR_TOKEN_RANGE;
    lo = hi = 0;
  }
  // this thread's first bias, with the words' loads
  int32_t tok = -1, before = -2;
  if (lo + static_cast<int32_t>(threadIdx.x) < hi) {
    tok = p.bias_tokens[lo + threadIdx.x];
    s_tok[threadIdx.x] = tok;
    s_val[threadIdx.x] = p.bias_values[lo + threadIdx.x];
    if (threadIdx.x > 0) before = p.bias_tokens[lo + threadIdx.x - 1];
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < nwords; i += kLogitThreads) {
    const int32_t w = word0 + i;
    const bool in_row = w >= 0;
    plane[i] = seen && in_row ? seen[w] : 0u;
    plane[kPlane + i] = seen && in_row ? seen[p.W + w] : 0u;
    plane[2 * kPlane + i] = mask ? in_row ? mask[w] : 0u : 0xffffffffu;
    plane[3 * kPlane + i] = 0u;
  }
  if (threadIdx.x == 0) s_total = s_listed = 0;
  const float rho = p.repetition ? p.repetition[row] : 1.f;
  const float freq = p.frequency ? p.frequency[row] : 0.f;
  const float pres = p.presence ? p.presence[row] : 0.f;
  const float temp = p.temperature ? p.temperature[row] : 0.f;
  const bool scale = temp > 0.f && temp != 1.f;
  const bool every = !p.inplace || scale;
  // quotients as products with the reciprocal in two parts (a tenth of the
  // instructions of a division); a temperature near an end of fp32 is taken 2^64 or
  // 2^-64 times, and its quotients again; such a repetition penalty divides
  const float after = !scale ? 1.f : temp < 1e-37f ? 0x1p64f : temp > 0x1p64f ? 0x1p-64f : 1.f;
  const Reciprocal inv(scale ? temp * after : 1.f), rinv(rho);
  const bool divide = !(rho > 0x1p-64f && rho < 0x1p64f);
  __syncthreads();
  for (int32_t e = lo + threadIdx.x; e < hi; e += kLogitThreads) {
    if (e != lo + static_cast<int32_t>(threadIdx.x)) {
      tok = p.bias_tokens[e];
      before = p.bias_tokens[e - 1];
    }
    if (tok < 0 || tok >= p.V || before >= tok) bad = MCP_DEVERR_TOKEN_RANGE;
    if (tok >= max(begin, 0) && tok < end)
      atomicOr(plane + 3 * kPlane + (tok >> 5) - word0, 1u << (tok & 31));
  }
  if (bad && part == 0 && p.err) atomicOr(p.err, bad);
  __syncthreads();

  // from here plane 0 has the tokens that a bias or penalty changes: seen or
  // biased, and allowed, without those of the neighbouring parts in a shifted
  // row's first and last word
  int total = 0;
  for (int i = threadIdx.x; i < nwords; i += kLogitThreads) {
    const int32_t v = 32 * (word0 + i);
    uint32_t own = plane[2 * kPlane + i];
    if (v < begin) own = own >> (begin - v) << (begin - v);
    if (end - v < 32) own &= (1u << (end - v)) - 1;
    const uint32_t any = plane[i] | plane[kPlane + i];
    plane[4 * kPlane + i] = any;
    const uint32_t changed = (any | plane[3 * kPlane + i]) & own;
    plane[i] = changed;
    total += __popc(changed);
  }
  total = __reduce_add_sync(0xffffffffu, total);
  if ((threadIdx.x & 31) == 0 && total) atomicAdd(&s_total, total);
  __syncthreads();

  const TI* in = static_cast<const TI*>(p.logits) + row * p.ld_in;
  TO* out = static_cast<TO*>(p.out) + row * p.ld_out;
  const int32_t* counts = p.counts + static_cast<int64_t>(id) * 32 * p.W;
  const int32_t first = (threadIdx.x >> 5) * 32 * kGroups * kVec + (threadIdx.x & 31) * kVec;
  const int turn = (begin + first) & 31;  // the place of a thread's groups in their words
  const uint32_t* bits0 = plane + ((begin + first) >> 5) - word0;

  // bits of the thread's group g of the tile at `base` (a multiple of 32 behind begin)
  auto bits_at = [&](int k, int32_t base, int g) {
    const uint32_t* w = bits0 + k * kPlane + ((base - begin) >> 5) + g * kVec;
    return kRows == kShifted ? __funnelshift_r(w[0], w[1], turn) : w[0] >> turn;
  };
  // tokens of the group that are in this part
  auto valid_at = [&](int32_t v) {
    const int32_t left = end - v;
    uint32_t m = left >= kVec ? kAll : left <= 0 ? 0u : (1u << left) - 1;
    if (kRows == kShifted && v < 0) m = m >> -v << -v;
    return m;
  };
  auto whole_tile = [&](int32_t base) { return base >= 0 && base + kLogitTile <= end; };
  // x / temperature, or the masked value
  auto finish = [&](float x) { return inv.times(x) * after; };
  auto put = [&](int32_t v, const float* x, uint32_t touch) {
    Vec<TO, kVec> y;
#pragma unroll
    for (int i = 0; i < kVec; ++i) y.v[i] = from_f<TO>(x[i]);
    if (touch == kAll) {
      *reinterpret_cast<Vec<TO, kVec>*>(out + v) = y;
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (touch >> i & 1) out[v + i] = y.v[i];
    }
  };
  // Request the logits of a tile that are not masked, process a tile.  In
  // place the tokens of plane 0 wait for their turn; elsewhere they are written
  // twice, whole vectors being cheaper than single tokens.  kEnds: the tile
  // may begin or end inside a group (a row's first and last).
  auto request = [&](int32_t base, int slot) {
    TI* to = ring + slot * kLogitTile + first;
    const TI* at = in + base + first;
    const bool whole = whole_tile(base);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (!whole && valid_at(base + first + g * 32 * kVec) != kAll) continue;
      if (mask && !(bits_at(2, base, g) & kAll)) continue;
      copy_async<kVec * sizeof(TI)>(to + g * 32 * kVec, at + g * 32 * kVec);
    }
  };
  auto process = [&](int32_t base, int slot, auto masked, auto ends) {
    constexpr bool kMask = decltype(masked)::value, kEnds = decltype(ends)::value;
    const TI* from = ring + slot * kLogitTile + first;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int32_t v = base + first + g * 32 * kVec;
      const uint32_t valid = kEnds ? valid_at(v) : kAll;
      if (kEnds && !valid) continue;
      uint32_t ok = kMask ? bits_at(2, base, g) : kAll;
      const uint32_t touch = p.inplace ? valid & ~bits_at(0, base, g) : valid;
      float x[kVec];
      if (kAsync && (!kEnds || valid == kAll)) {
        const Vec<TI, kVec> q = *reinterpret_cast<const Vec<TI, kVec>*>(from + g * 32 * kVec);
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = to_f(q.v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = touch & ok & 1u << i ? to_f(in[v + i]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        x[i] = finish(x[i]);
        // what was not requested is masked
        if (kMask) x[i] = ok & 1u << i ? x[i] : -INFINITY;
      }
      put(v, x, touch);
    }
  };
  using std::false_type;
  using std::true_type;
  if (every) {
    if constexpr (kAsync) {
#pragma unroll
      for (int s = 0; s < kSlots - 1; ++s) {
        if (begin + s * kLogitTile < end) request(begin + s * kLogitTile, s);
        copy_commit();
      }
    }
    int slot = 0;
    for (int32_t base = begin; base < end; base += kLogitTile) {
      if constexpr (kAsync) {
        const int32_t ahead = base + (kSlots - 1) * kLogitTile;
        if (ahead < end) request(ahead, slot == 0 ? kSlots - 1 : slot - 1);
        copy_commit();
        copy_wait<kSlots - 1>();
      }
      if (!whole_tile(base)) process(base, slot, true_type(), true_type());
      else if (mask) process(base, slot, true_type(), false_type());
      else process(base, slot, false_type(), false_type());
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }
  } else if (mask) {
    // in place, as they are: only the masked tokens are written
    float x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = -INFINITY;
    for (int32_t base = begin; base < end; base += kLogitTile) {
#pragma unroll 2
      for (int g = 0; g < kGroups; ++g) {
        const int32_t v = base + first + g * 32 * kVec;
        const uint32_t touch = valid_at(v) & ~bits_at(2, base, g);
        if (touch) put(v, x, touch);
      }
    }
  }

  // The tokens of plane 0, listed in shared memory (the ring is done with, and
  // the barrier orders the pass's writes before these), so
  // that every thread has as many as the next: a branch in the pass would cost
  // every warp that has one of them.
  uint16_t* list = reinterpret_cast<uint16_t*>(lsmem);
  constexpr int kList = kLogitRing<TI> / 2;  // entries
  const int lane = threadIdx.x & 31;
  const int window = s_total <= kList ? nwords : kList / 32;  // words whose tokens the list has room for
  for (int w0 = 0; w0 < nwords && s_total > 0; w0 += window) {
    __syncthreads();  // the ring, and the list before
    if (w0 > 0) {
      if (threadIdx.x == 0) s_listed = 0;
      __syncthreads();
    }
    const int w1 = min(nwords, w0 + window);
    for (int w8 = w0 + (threadIdx.x >> 5); w8 < w1; w8 += kLogitThreads) {
      const int w = w8 + kLogitThreads / 32 * lane;
      const uint32_t m = w < w1 ? plane[w] : 0u;
      const int n = __popc(m);
      if (!__any_sync(0xffffffffu, n)) continue;
      int at = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += u;
      }
      int base = 0;
      if (lane == 31) base = atomicAdd(&s_listed, at);
      at += __shfl_sync(0xffffffffu, base, 31) - n;
      // words of a few tokens each by its lane, full ones by the warp; a warp's
      // words are not neighbours, as frequent tokens are: full words that met in
      // one warp cost 64 rows 2 us
      constexpr int kFew = 8;
      if (n <= kFew) {
        int a = at;
        for (uint32_t x = m; x; x &= x - 1) list[a++] = static_cast<uint16_t>(32 * w + __ffs(x) - 1);
      }
      for (uint32_t full = __ballot_sync(0xffffffffu, n > kFew); full; full &= full - 1) {
        const int src = __ffs(full) - 1;
        const uint32_t x = __shfl_sync(0xffffffffu, m, src);
        const int a = __shfl_sync(0xffffffffu, at, src);
        if (x >> lane & 1) list[a + __popc(x & ((1u << lane) - 1))] = static_cast<uint16_t>(32 * (w8 + kLogitThreads / 32 * src) + lane);
      }
    }
    __syncthreads();
    const int listed = s_listed;
    constexpr int kAtOnce = 4;  // tokens of a thread whose loads are in flight together
    for (int e0 = threadIdx.x; e0 < listed; e0 += kAtOnce * kLogitThreads) {
      int k[kAtOnce], sh[kAtOnce];
      int32_t n[kAtOnce];
      TI q[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int e = e0 + j * kLogitThreads;
        k[j] = -1;
        n[j] = 0;
        if (e >= listed) continue;
        k[j] = list[e] >> 5;
        sh[j] = list[e] & 31;
        const int32_t v = 32 * (word0 + k[j]) + sh[j];
        q[j] = in[v];
        if (plane[kPlane + k[j]] >> sh[j] & 1) n[j] = counts[v];
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (k[j] < 0) continue;
        const int32_t v = 32 * (word0 + k[j]) + sh[j];
        float x = to_f(q[j]);
        bool had = true;
        if (plane[3 * kPlane + k[j]] >> sh[j] & 1) {
          x += hi - lo <= kLogitThreads ? find_bias(s_tok, s_val, 0, hi - lo, v)
                                        : find_bias(p.bias_tokens, p.bias_values, lo, hi, v);
          had = plane[4 * kPlane + k[j]] >> sh[j] & 1;
        }
        if (had) x = x <= 0.f ? x * rho : divide ? __fdiv_rn(x, rho) : rinv.times(x);
        if (n[j] > 0) x = x - __fmul_rn(freq, static_cast<float>(n[j])) - pres;
        out[v] = from_f<TO>(finish(x));
      }
    }
  }
}

template <typename TI, typename TO, int kRows>
int logits_rows(const LogitArgs& a, cudaStream_t st) {
  constexpr auto kernel = process_logits_kernel<TI, TO, kRows>;
  if (const int e = allow_smem<kernel>(kLogitSmem<TI>)) return e;
  const int64_t grid = static_cast<int64_t>(a.rows) * a.parts;
  kernel<<<static_cast<unsigned>(grid), kLogitThreads, kLogitSmem<TI>, st>>>(a);
  return static_cast<int>(cudaGetLastError());
}

template <typename TI, typename TO>
int logits_launch(const LogitArgs& a, cudaStream_t st) {
  // the same tokens stand on vector boundaries of both, in every row
  const uintptr_t in = reinterpret_cast<uintptr_t>(a.logits), out = reinterpret_cast<uintptr_t>(a.out);
  const bool vec = (in / sizeof(TI) - out / sizeof(TO)) % 4 == 0 && (a.ld_in - a.ld_out) % 4 == 0;
  const bool even = (out / sizeof(TO)) % 4 == 0 && a.ld_out % 4 == 0;
  return vec && even ? logits_rows<TI, TO, kWhole>(a, st)
         : vec       ? logits_rows<TI, TO, kShifted>(a, st)
                     : logits_rows<TI, TO, kSingle>(a, st);
}

}  // namespace

int launch_update_token_counts(const int32_t* request_ids, int32_t num_rows,
                               const int32_t* tokens, int32_t num_tokens,
                               const int32_t* cu_tokens, int32_t* seen, int32_t* counts,
                               int32_t num_requests, int32_t vocab_size, int32_t flags,
                               int32_t* error_word, void* stream) {
  CountArgs a;
  a.ids = request_ids;
  a.tokens = tokens;
  a.cu = cu_tokens;
  a.seen = seen;
  a.counts = counts;
  a.err = error_word;
  a.rows = num_rows;
  a.n = num_tokens;
  a.R = num_requests;
  a.V = vocab_size;
  a.W = (vocab_size + 31) / 32;
  a.prompt = flags & MCP_COUNT_PROMPT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (flags & MCP_COUNT_RESET) {
    const int64_t blocks = (static_cast<int64_t>(num_rows) * a.W + kCountThreads - 1) / kCountThreads;
    const int64_t cap = 16LL * step_num_sms();
    clear_counts_kernel<<<static_cast<unsigned>(blocks < cap ? blocks : cap), kCountThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  if (num_tokens == 0) return 0;
  const bool beside = flags & MCP_COUNT_RESET;  // begins while the rows are cleared
  if (cu_tokens && num_tokens >= kMarkTokens && num_tokens / num_rows >= (a.prompt ? kMarkRow : kCountRow)) {
    const int32_t sms = step_num_sms();
    int32_t chunk = ((num_tokens + sms - 1) / sms + kMarkThreads - 1) / kMarkThreads * kMarkThreads;
    if (chunk < 2 * kMarkThreads) chunk = 2 * kMarkThreads;
    const int32_t words = ((vocab_size < kMapTokens ? vocab_size : kMapTokens) + 31) / 32;
    return launch_beside(mark_texts_kernel, beside, (num_tokens - 1) / chunk + 1, kMarkThreads, 4 * words, st, a,
                         chunk);
  }
  return launch_beside(add_tokens_kernel, beside, (num_tokens - 1) / kCountThreads + 1, kCountThreads, 0, st, a);
}

int launch_process_logits(const mcp_logits_desc& d, const mcp_logits_tensors& t,
                          int32_t* error_word, void* stream) {
  LogitArgs a;
  a.logits = t.logits;
  a.out = t.out;
  a.ids = t.request_ids;
  a.seen = t.seen;
  a.counts = t.counts;
  a.temperature = t.temperature;
  a.repetition = t.repetition_penalty;
  a.frequency = t.frequency_penalty;
  a.presence = t.presence_penalty;
  a.bias_offsets = t.bias_offsets;
  a.bias_tokens = t.bias_tokens;
  a.bias_values = t.bias_values;
  a.mask = t.mask;
  a.mask_rows = t.mask_rows;
  a.err = error_word;
  a.ld_in = d.logits_stride;
  a.ld_out = d.out_stride;
  a.rows = d.num_rows;
  a.V = d.vocab_size;
  a.W = (d.vocab_size + 31) / 32;
  a.R = d.num_requests;
  a.num_bias = d.num_biases;
  a.num_masks = d.num_masks;
  // a CTA reads its row's parameters, bits and biases once for several tiles
  // where there are enough for six CTAs on every SM (64 rows of bf16 in place, 2000
  // seen tokens a row, no biases or masks: 8.3 us; for three and four 8.8, for eight
  // 9.1; of fp32, of which four CTAs fit an SM, 10.0, 8.5 and 9.0)
  const int64_t row_tiles = (d.vocab_size + 3LL + kLogitTile - 1) / kLogitTile;  // shifted by up to 3
  const int64_t places = 6LL * step_num_sms();
  int64_t tiles = (row_tiles * d.num_rows + places - 1) / places;
  tiles = tiles < 1 ? 1 : tiles > kLogitMaxTiles ? kLogitMaxTiles : tiles;
  tiles = tiles > row_tiles ? row_tiles : tiles;
  a.tiles = static_cast<int32_t>(tiles);
  a.parts = static_cast<int32_t>((row_tiles + tiles - 1) / tiles);
  a.inplace = t.logits == t.out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = d.dtype == d.out_dtype;
  if (d.dtype == MCP_DTYPE_BF16)
    return same ? logits_launch<__nv_bfloat16, __nv_bfloat16>(a, st)
                : logits_launch<__nv_bfloat16, float>(a, st);
  if (d.dtype == MCP_DTYPE_FP16)
    return same ? logits_launch<__half, __half>(a, st) : logits_launch<__half, float>(a, st);
  return logits_launch<float, float>(a, st);
}

}  // namespace mcp
