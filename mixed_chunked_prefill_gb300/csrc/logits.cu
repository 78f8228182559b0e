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
  const int64_t total = static_cast<int64_t>(p.rows) * p.W;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCountThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kCountThreads) {
    const int32_t r = static_cast<int32_t>(i / p.W), w = static_cast<int32_t>(i - static_cast<int64_t>(r) * p.W);
    const int32_t id = p.ids[r];
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

// Adding and marking are atomic, so the result does not depend on the order and
// a request may stand in several rows; a mark that is already there is only
// read (text repeats few words very often).  A thread takes kPer neighbouring
// tokens whose loads are in flight together; the row of a CTA's first token is
// looked up once, and a token looks its own up only behind that row's end.
// Repeats within a CTA's part of that row are dropped by a bitmap in shared
// memory: a cleared row whose most frequent tokens were all marked at once took
// 20 us longer for 64 prompts of 24000 tokens, one word taking thousands of
// atomics.
constexpr int kFilterTokens = 1 << 17;  // 16 KB; tokens from there on are not filtered

template <int kPer>
__global__ void __launch_bounds__(kCountThreads) add_tokens_kernel(const CountArgs p) {
  __shared__ int32_t s_row, s_end;
  __shared__ __align__(16) uint32_t filter[kPer > 1 ? kFilterTokens / 32 : 4];
  const int32_t c0 = blockIdx.x * (kCountThreads * kPer);
  auto find = [&](int32_t i) {  // first row that ends behind token i
    int32_t lo = 0, hi = p.rows;
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if (p.cu[mid + 1] <= i) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  const int32_t i0 = c0 + threadIdx.x * kPer;
  int32_t tok[kPer];
  // whole vectors where the tokens are aligned; behind num_tokens nothing is read
  const bool vec = kPer % 4 == 0 && (reinterpret_cast<uintptr_t>(p.tokens) & 15) == 0 && i0 + kPer <= p.n;
  if constexpr (kPer % 4 == 0) {
    if (vec) {
#pragma unroll
      for (int k = 0; k < kPer; k += 4) {
        const int4 q = *reinterpret_cast<const int4*>(p.tokens + i0 + k);
        tok[k] = q.x, tok[k + 1] = q.y, tok[k + 2] = q.z, tok[k + 3] = q.w;
      }
    }
  }
  if (!vec) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) tok[k] = i0 + k < p.n ? p.tokens[i0 + k] : -1;
  }
  int32_t row0 = 0, end0 = 0;
  if (p.cu && kPer > 1) {
    const int words = (min(p.V, kFilterTokens) + 127) / 128;
    for (int w = threadIdx.x; w < words; w += kCountThreads)
      reinterpret_cast<uint4*>(filter)[w] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) {
      s_row = find(c0);
      s_end = s_row < p.rows ? p.cu[s_row + 1] : 0;
    }
    __syncthreads();
    row0 = s_row;
    end0 = s_end;
    if (row0 < p.rows && p.cu[row0] > c0) end0 = 0;  // tokens before the first row
  }
  int bad = 0;
  int32_t* word[kPer];
  uint32_t had[kPer];
  int32_t id = -1, last = -2;  // request row of the row `last`
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int32_t i = i0 + k;
    word[k] = nullptr;
    had[k] = 0xffffffffu;
    if (i >= p.n) continue;
    int32_t row = i;
    if (p.cu) {
      row = row0;
      if (i >= end0) {
        row = find(i);
        if (row < p.rows && p.cu[row] > i) row = p.rows;
      }
    }
    if (row != last) id = row < p.rows ? p.ids[row] : -1;
    last = row;
    if (id >= p.R) {
      bad |= MCP_DEVERR_REQUEST;
    } else if (id >= 0 && tok[k] >= p.V) {
      bad |= MCP_DEVERR_TOKEN_RANGE;
    } else if (id >= 0 && tok[k] >= 0) {
      const uint32_t bit = 1u << (tok[k] & 31);
      const bool repeat = kPer > 1 && p.cu && row == row0 && i < end0 && tok[k] < kFilterTokens &&
                          (atomicOr(filter + (tok[k] >> 5), bit) & bit);
      if (!repeat) {
        word[k] = p.seen + (static_cast<int64_t>(id) * 2 + (p.prompt ? 0 : 1)) * p.W + (tok[k] >> 5);
        had[k] = *reinterpret_cast<volatile uint32_t*>(word[k]);
      }
      if (!p.prompt) atomicAdd(p.counts + static_cast<int64_t>(id) * 32 * p.W + tok[k], 1);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const uint32_t bit = 1u << (tok[k] & 31);
    if (word[k] && !(had[k] & bit)) atomicOr(reinterpret_cast<unsigned int*>(word[k]), bit);
  }
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
constexpr int kLogitMaxTiles = 8;               // tiles of one CTA

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

// The bias of token `tok`, which has one: entries [lo, hi) in rising order.
__device__ __noinline__ float find_bias(const LogitArgs& p, int32_t lo, int32_t hi, int32_t tok) {
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (p.bias_tokens[mid] <= tok) lo = mid;
    else hi = mid;
  }
  return p.bias_tokens[lo] == tok ? p.bias_values[lo] : 0.f;
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
__device__ __forceinline__ void prefetch(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
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
// are listed and taken afterwards, one a thread.
enum LogitRows { kWhole, kShifted, kSingle };

constexpr int kLogitWords = kLogitMaxTiles * kLogitTile / 32;  // of a plane, in a part
// tiles of logits in flight and CTAs an SM: 32 KB and 4 (16 bits), 48 KB and 3 (fp32)
template <typename T>
constexpr int kLogitSlots = sizeof(T) == 2 ? 4 : 3;
template <typename T>
constexpr int kLogitRing = kLogitSlots<T> * kLogitTile * static_cast<int>(sizeof(T));
template <typename T>
constexpr int kLogitSmem = 4 * 4 * (kLogitWords + 2) + kLogitRing<T>;

template <typename TI, typename TO, int kRows>
__global__ void __launch_bounds__(kLogitThreads, sizeof(TI) == 2 ? 4 : 3) process_logits_kernel(const LogitArgs p) {
  constexpr int kVec = kRows == kSingle ? 1 : 4;
  constexpr int kGroups = kLogitTile / kLogitThreads / kVec;  // of a thread and tile
  constexpr uint32_t kAll = (1u << kVec) - 1;
  constexpr bool kAsync = kVec * sizeof(TI) >= 4;
  constexpr int kSlots = kLogitSlots<TI>;
  extern __shared__ __align__(16) unsigned char lsmem[];
  TI* ring = reinterpret_cast<TI*>(lsmem);
  uint32_t* plane = reinterpret_cast<uint32_t*>(lsmem + kLogitRing<TI>);  // prompt, sampled, allowed, biased
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
  const float rho = p.repetition ? p.repetition[row] : 1.f;
  const float freq = p.frequency ? p.frequency[row] : 0.f;
  const float pres = p.presence ? p.presence[row] : 0.f;
  const float temp = p.temperature ? p.temperature[row] : 0.f;
  const bool scale = temp > 0.f && temp != 1.f;
  const bool every = !p.inplace || scale;
  // quotients as products: one rounding more, a tenth of the instructions;
  // divisors whose reciprocal overflows divide
  const float inv = scale ? 1.f / temp : 1.f, rinv = 1.f / rho;
  const bool divide = inv > 3.4e38f || rinv > 3.4e38f;
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
  // row's first and last word; the counts of the sampled ones are on their way to L2
  for (int i = threadIdx.x; i < nwords; i += kLogitThreads) {
    const int32_t v = 32 * (word0 + i);
    uint32_t own = plane[2 * kPlane + i];
    if (v < begin) own = own >> (begin - v) << (begin - v);
    if (end - v < 32) own &= (1u << (end - v)) - 1;
    const uint32_t had = plane[kPlane + i] & own;
    plane[i] = (plane[i] | plane[kPlane + i] | plane[3 * kPlane + i]) & own;
    const int32_t* c = p.counts + (static_cast<int64_t>(id) * p.W + word0 + i) * 32;
    for (uint32_t m = had; m; m &= m - 1) prefetch(c + __ffs(m) - 1);
  }
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
  auto finish = [&](float x) { return divide ? scale ? __fdiv_rn(x, temp) : x : x * inv; };
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
  constexpr int kListWords = 2 * kLogitThreads;  // 16384 tokens: 32 KB of list
  __shared__ int32_t warp_sum[kLogitThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w0 = 0; w0 < nwords; w0 += kListWords) {
    const int i = w0 + 2 * threadIdx.x;
    const uint32_t a = i < nwords ? plane[i] : 0u, b = i + 1 < nwords ? plane[i + 1] : 0u;
    const int mine = __popc(a) + __popc(b);
    int at = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += u;
    }
    __syncthreads();  // the ring, and the list before
    if (lane == 31) warp_sum[warp] = at;
    __syncthreads();
    int total = 0;
    at -= mine;
#pragma unroll
    for (int k = 0; k < kLogitThreads / 32; ++k) {
      if (k < warp) at += warp_sum[k];
      total += warp_sum[k];
    }
    for (uint32_t m = a; m; m &= m - 1) list[at++] = static_cast<uint16_t>(64 * threadIdx.x + __ffs(m) - 1);
    for (uint32_t m = b; m; m &= m - 1) list[at++] = static_cast<uint16_t>(64 * threadIdx.x + 31 + __ffs(m));
    __syncthreads();
    constexpr int kAtOnce = 4;  // tokens of a thread whose loads are in flight together
    for (int e0 = threadIdx.x; e0 < total; e0 += kAtOnce * kLogitThreads) {
      int k[kAtOnce], sh[kAtOnce];
      int32_t n[kAtOnce];
      TI q[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int e = e0 + j * kLogitThreads;
        k[j] = -1;
        n[j] = 0;
        if (e >= total) continue;
        k[j] = w0 + (list[e] >> 5);
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
          x += find_bias(p, lo, hi, v);
          had = seen && (seen[word0 + k[j]] | seen[p.W + word0 + k[j]]) >> sh[j] & 1;
        }
        if (had) x = x <= 0.f ? x * rho : divide ? __fdiv_rn(x, rho) : x * rinv;
        if (n[j] > 0) x = x - __fmul_rn(freq, static_cast<float>(n[j])) - pres;
        out[v] = from_f<TO>(finish(x));
      }
    }
  }
}

template <typename TI, typename TO, int kRows>
int logits_rows(const LogitArgs& a, cudaStream_t st) {
  if (const int e = allow_smem<process_logits_kernel<TI, TO, kRows>>(kLogitSmem<TI>)) return e;
  const int64_t grid = static_cast<int64_t>(a.rows) * a.parts;
  process_logits_kernel<TI, TO, kRows>
      <<<static_cast<unsigned>(grid), kLogitThreads, kLogitSmem<TI>, st>>>(a);
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
  // eight tokens a thread once they fill the SMs
  constexpr int kMany = 8;
  if (num_tokens >= kMany * kCountThreads * step_num_sms()) {
    constexpr int chunk = kMany * kCountThreads;
    add_tokens_kernel<kMany><<<(num_tokens - 1) / chunk + 1, kCountThreads, 0, st>>>(a);
  } else if (num_tokens > 0) {
    add_tokens_kernel<1><<<(num_tokens - 1) / kCountThreads + 1, kCountThreads, 0, st>>>(a);
  }
  return static_cast<int>(cudaGetLastError());
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
  // a CTA reads its row's parameters, bits and biases once for several tiles:
  // as few CTAs as find a place on the SMs together (a second wave would wait
  // for its own first loads again), up to the tiles that shared memory has bits for
  const int64_t row_tiles = (d.vocab_size + 3LL + kLogitTile - 1) / kLogitTile;  // shifted by up to 3
  const int64_t places = (d.dtype == MCP_DTYPE_FP32 ? 3LL : 4LL) * step_num_sms();
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
