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

// One thread a token.  Adding and marking are atomic, so the result does not
// depend on the order and a request may stand in several rows; a mark that is
// already there is only read (text repeats few words very often).
__global__ void __launch_bounds__(kCountThreads) add_tokens_kernel(const CountArgs p) {
  const int32_t i = blockIdx.x * kCountThreads + threadIdx.x;
  int bad = 0;
  if (i < p.n) {
    int32_t row = i;
    if (p.cu) {
      int32_t lo = 0, hi = p.rows;  // first row that ends behind token i
      while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (p.cu[mid + 1] <= i) lo = mid + 1;
        else hi = mid;
      }
      row = lo < p.rows && p.cu[lo] <= i ? lo : -1;
    }
    const int32_t id = row < 0 ? -1 : p.ids[row];
    const int32_t tok = p.tokens[i];
    if (id >= p.R) {
      bad = MCP_DEVERR_REQUEST;
    } else if (id >= 0 && tok >= p.V) {
      bad = MCP_DEVERR_TOKEN_RANGE;
    } else if (id >= 0 && tok >= 0) {
      int32_t* word = p.seen + (static_cast<int64_t>(id) * 2 + (p.prompt ? 0 : 1)) * p.W + (tok >> 5);
      const uint32_t bit = 1u << (tok & 31);
      if (!(*reinterpret_cast<volatile uint32_t*>(word) & bit))
        atomicOr(reinterpret_cast<unsigned int*>(word), bit);
      if (!p.prompt) atomicAdd(p.counts + static_cast<int64_t>(id) * 32 * p.W + tok, 1);
    }
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
  int32_t rows, V, W, R, num_bias, num_masks, tiles, inplace;
};

constexpr int kLogitThreads = 256;
constexpr int kLogitTile = 8 * kLogitThreads;  // tokens of one row a CTA takes

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

template <typename T>
struct alignas(8 * sizeof(T) < 16 ? 8 * sizeof(T) : 16) Vec8 {
  T v[8];
};

struct RowParams {
  float rho, freq, pres, temp;
};

__device__ __forceinline__ float process(float x, float bias, bool seen, int32_t count, bool allow,
                                         const RowParams& r) {
  x += bias;
  if (seen) x = x > 0.f ? __fdiv_rn(x, r.rho) : x * r.rho;
  if (count > 0) x = x - __fmul_rn(r.freq, static_cast<float>(count)) - r.pres;
  if (r.temp > 0.f) x = __fdiv_rn(x, r.temp);
  return allow ? x : -INFINITY;
}

// kVec 8: a thread takes 8 neighbouring tokens with 16-byte accesses (rows
// that start on 16 bytes).  kVec 1: rows that start anywhere (an odd
// vocabulary); a warp takes 32 neighbouring tokens at a time.
template <typename TI, typename TO, int kVec>
__global__ void __launch_bounds__(kLogitThreads) process_logits_kernel(const LogitArgs p) {
  __shared__ float sbias[kLogitTile];
  const int32_t row = blockIdx.x / p.tiles, tile = blockIdx.x - row * p.tiles;
  const int32_t v0 = tile * kLogitTile;
  const int32_t id = p.ids ? p.ids[row] : 0;
  int32_t mrow = !p.mask ? -1 : p.mask_rows ? p.mask_rows[row] : row;
  if (id < 0) return;  // padding: the row stays as it was
  if ((p.ids && id >= p.R) || mrow >= p.num_masks) {
    if (tile == 0 && threadIdx.x == 0 && p.err) atomicOr(p.err, MCP_DEVERR_REQUEST);
    return;
  }
  RowParams r;
  r.rho = p.repetition ? p.repetition[row] : 1.f;
  r.freq = p.frequency ? p.frequency[row] : 0.f;
  r.pres = p.presence ? p.presence[row] : 0.f;
  r.temp = p.temperature ? p.temperature[row] : 0.f;
  const bool every = !p.inplace || (r.temp > 0.f && r.temp != 1.f);

  // biases of this tile
  bool biased = false;
  if (p.bias_offsets) {
    int32_t lo = p.bias_offsets[row], hi = p.bias_offsets[row + 1];
    int bad = 0;
    if (lo < 0 || hi < lo || hi > p.num_bias) {
      bad = MCP_DEVERR_TOKEN_RANGE;
      lo = hi = 0;
    }
    bool mine = false;
    for (int32_t e = lo + threadIdx.x; e < hi; e += kLogitThreads) {
      const int32_t tok = p.bias_tokens[e];
      if (tok < 0 || tok >= p.V || (e > lo && p.bias_tokens[e - 1] >= tok)) bad = MCP_DEVERR_TOKEN_RANGE;
      mine |= tok >= v0 && tok < v0 + kLogitTile;
    }
    if (bad && tile == 0 && p.err) atomicOr(p.err, bad);
    biased = __syncthreads_or(mine);
    if (biased) {
      for (int i = threadIdx.x; i < kLogitTile; i += kLogitThreads) sbias[i] = 0.f;
      __syncthreads();
      for (int32_t e = lo + threadIdx.x; e < hi; e += kLogitThreads) {
        const int32_t tok = p.bias_tokens[e];
        if (tok >= v0 && tok < v0 + kLogitTile && tok < p.V) sbias[tok - v0] = p.bias_values[e];
      }
      __syncthreads();
    }
  }
  const TI* in = static_cast<const TI*>(p.logits) + row * p.ld_in;
  TO* out = static_cast<TO*>(p.out) + row * p.ld_out;
  const uint32_t* seen = reinterpret_cast<const uint32_t*>(p.seen) + static_cast<int64_t>(id) * 2 * p.W;
  const uint32_t* mask =
      mrow < 0 ? nullptr : reinterpret_cast<const uint32_t*>(p.mask) + static_cast<int64_t>(mrow) * p.W;
  const int32_t* counts = p.counts + static_cast<int64_t>(id) * 32 * p.W;

  if constexpr (kVec == 8) {
    const int32_t t = 8 * threadIdx.x, v = v0 + t;
    if (v >= p.V) return;
    const int32_t w = v >> 5, sh = v & 31;
    const int32_t n = min(8, p.V - v);
    const uint32_t valid = (1u << n) - 1;
    uint32_t pr = 0, ou = 0, al = 0xff;
    if (p.ids) {
      pr = seen[w] >> sh & 0xff;
      ou = seen[p.W + w] >> sh & 0xff;
    }
    if (mrow >= 0) al = mask[w] >> sh & 0xff;
    uint32_t touch = (every ? 0xffu : pr | ou | ~al) & valid;
    float bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bias[i] = biased ? sbias[t + i] : 0.f;
      if (bias[i] != 0.f) touch |= 1u << i;
    }
    touch &= valid;
    if (!touch) return;
    float x[8];
    if (touch & al) {
      if (n == 8) {
        const Vec8<TI> q = *reinterpret_cast<const Vec8<TI>*>(in + v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f(q.v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? to_f(in[v + i]) : 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    int32_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (ou & al) {
      const int4 a = *reinterpret_cast<const int4*>(counts + v);
      const int4 b = *reinterpret_cast<const int4*>(counts + v + 4);
      c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
      c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
    }
    const uint32_t had = pr | ou;
    Vec8<TO> y;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y.v[i] = from_f<TO>(process(x[i], bias[i], had >> i & 1, ou >> i & 1 ? c[i] : 0, al >> i & 1, r));
    if (n == 8 && (every || !p.inplace)) {
      *reinterpret_cast<Vec8<TO>*>(out + v) = y;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (touch >> i & 1) out[v + i] = y.v[i];
    }
  } else {
    const int lane = threadIdx.x & 31;
    const int32_t t = (threadIdx.x >> 5) * 256 + lane;
    float x[8];
    int32_t c[8];
    uint32_t bits[8];  // 1 seen, 2 allowed, 4 touched
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t v = v0 + t + 32 * i, w = v >> 5;
      x[i] = 0.f;
      c[i] = 0;
      bits[i] = 0;
      if (v >= p.V) continue;
      uint32_t pr = 0, ou = 0, al = 1;
      if (p.ids) {
        pr = seen[w] >> lane & 1;
        ou = seen[p.W + w] >> lane & 1;
      }
      if (mrow >= 0) al = mask[w] >> lane & 1;
      const bool b = biased && sbias[t + 32 * i] != 0.f;
      bits[i] = (pr | ou) | al << 1 | (every || pr || ou || !al || b ? 4 : 0);
      if (al && bits[i] & 4) x[i] = to_f(in[v]);
      if (al && ou) c[i] = counts[v];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(bits[i] & 4)) continue;
      out[v0 + t + 32 * i] = from_f<TO>(process(x[i], biased ? sbias[t + 32 * i] : 0.f, bits[i] & 1,
                                                c[i], bits[i] & 2, r));
    }
  }
}

template <typename TI, typename TO>
int logits_launch(const LogitArgs& a, cudaStream_t st) {
  const int64_t grid = static_cast<int64_t>(a.rows) * a.tiles;
  const bool vec =
      ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0 &&
      a.ld_in * sizeof(TI) % 16 == 0 && a.ld_out * sizeof(TO) % 16 == 0;
  if (vec)
    process_logits_kernel<TI, TO, 8><<<static_cast<unsigned>(grid), kLogitThreads, 0, st>>>(a);
  else
    process_logits_kernel<TI, TO, 1><<<static_cast<unsigned>(grid), kLogitThreads, 0, st>>>(a);
  return static_cast<int>(cudaGetLastError());
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
  if (num_tokens > 0)
    add_tokens_kernel<<<(num_tokens + kCountThreads - 1) / kCountThreads, kCountThreads, 0, st>>>(a);
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
  a.tiles = (d.vocab_size + kLogitTile - 1) / kLogitTile;
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
