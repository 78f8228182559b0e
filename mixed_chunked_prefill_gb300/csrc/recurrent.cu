// The recurrent layers of a step over the packed stream: the short causal
// convolution and the selective state space scan, each segment continued from
// the state of its request and leaving its state for the next step.
//
// The stream is the one the mixed attention runs on ([W] "Flash Attention 的
// varlen 接口": decodes and chunks are segments of different lengths; the
// segment has history when seqlens_k counts more than its own tokens), so a
// decode is a segment of one token and a continued chunk starts from its
// request's state.  A segment's state is read and written by the one warp (or
// thread) that owns its channels; only a long segment that the scan cuts hands its
// states from piece to piece, through the workspace.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

// ------------------------------------------------------------------ elements
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float* f);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f);
template <>
__device__ __forceinline__ uint4 pack8<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack8<__half>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void unpack4(const uint2& v, float* f) {
  float g[8];
  unpack8<T>(make_uint4(v.x, v.y, 0u, 0u), g);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = g[i];
}

template <typename T>
__device__ __forceinline__ uint2 pack4(const float* f) {
  const float g[8] = {f[0], f[1], f[2], f[3], 0.f, 0.f, 0.f, 0.f};
  const uint4 v = pack8<T>(g);
  return make_uint2(v.x, v.y);
}
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

using f32x2 = unsigned long long;  // two fp32 lanes in one register pair
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// the smaller; NaN if one is
__device__ __forceinline__ float least(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the larger; NaN if one is
__device__ __forceinline__ float greatest(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ f32x2 ex2x2(f32x2 v) {
  float a, b;
  unpack2(v, a, b);
  return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// v / (1 + exp(-v)), exp as the square of its root and the sum taken 2^-20 times, so
// that neither overflows and the reciprocal is no subnormal (flushed to 0) before v
// = -101, where the quotient is below what bf16 holds.
__device__ __forceinline__ float silu(float v) {
  const float root = ex2(-0.5f * kLog2e * v);
  return v * (rcp(fmaf(0x1p-20f * root, root, 0x1p-20f)) * 0x1p-20f);
}

// ------------------------------------------------------------------ segments
struct Segments {
  const int32_t* ids;
  const int32_t* cu;
  const int32_t* sk;
  int32_t S, T, R;
  int32_t* err;
  int32_t sms;  // of the device
};

constexpr int kShortTokens = 4;  // short segments: decodes, a few speculated tokens

// Segment s's tokens [q0, q1), request row and whether it continues a state;
// id < 0: padding, or a segment the check reports (it is then left out).
struct Segment {
  int32_t q0, q1, id, old;
};
__device__ __forceinline__ Segment read_segment(const Segments& g, int32_t s) {
  Segment x;
  x.q0 = g.cu[s];
  x.q1 = g.cu[s + 1];
  x.id = g.ids[s];
  x.old = g.sk[s] > x.q1 - x.q0;
  // compared as they are: the difference of wild bounds leaves 32 bits
  if (x.q0 < 0 || x.q1 < x.q0 || x.q1 > g.T || x.id >= g.R) x.id = -1;
  return x;
}

// One CTA of a call (of the scan's last launch) looks the metadata over: segments outside the stream,
// request rows outside the state, a request in two segments that have tokens
// (its state would be written twice).  Rows are marked in windows of 32768.
__device__ void check_segments(const Segments& g) {
  constexpr int32_t kWindow = 1 << 15;
  __shared__ uint32_t seen[kWindow / 32];
  int32_t bad = 0;
  for (int32_t w0 = 0; w0 < g.R; w0 += kWindow) {
    __syncthreads();
    for (int i = threadIdx.x; i < kWindow / 32; i += blockDim.x) seen[i] = 0;
    __syncthreads();
    for (int32_t s = threadIdx.x; s < g.S; s += blockDim.x) {
      const int32_t q0 = g.cu[s], q1 = g.cu[s + 1], id = g.ids[s];
      if (q0 < 0 || q1 < q0 || q1 > g.T || (s == 0 && q0 != 0) || g.sk[s] < q1 - q0)
        bad |= MCP_DEVERR_SEGMENT;
      if (id >= g.R) bad |= MCP_DEVERR_REQUEST;
      const int32_t r = id - w0;
      if (id < 0 || q1 <= q0 || r < 0 || r >= kWindow) continue;
      const uint32_t bit = 1u << (r & 31);
      if (atomicOr(seen + (r >> 5), bit) & bit) bad |= MCP_DEVERR_REQUEST;
    }
  }
  if (bad && g.err) atomicOr(g.err, bad);
}

// -------------------------------------------------------------- convolution
// y[t] = act(b + sum_k w[k] v[t - K + 1 + k]) per channel, v being the
// segment's inputs and, before them, the K - 1 inputs its request kept.
//
// Each input is read once and each output written once.  Segments of at most 4
// tokens (decodes) get a CTA per two of them and 512 channels: the kept inputs
// and first tokens of both are requested at once, which is what their few
// microseconds consist of (1000 decodes of 8192 channels: 28 us, 4.7 TB/s; one,
// three or four segments a CTA 30, 32 and 34 us; 256 decodes: 8.8 us).  The
// tokens of longer segments are dealt in runs of TT (8192 tokens of 8192
// channels: 51 us, 5.2 TB/s; runs of 32 50, but 2048 tokens and 64 decodes 18.6
// instead of 18.2): a thread carries the K - 1 last inputs of 4 channels in
// registers, so only the first tokens of a run read inputs again (HBM-bound; 64
// registers, so that 32 warps an SM have 4 loads of 8 bytes in flight a thread; with
// four taps 64 bytes a thread are spilled for that).  The run that holds a
// segment's first token also takes its next K - 2 (even past its end: those still
// need the kept inputs) and writes the new kept inputs, so nobody else reads or
// writes that state.
struct ConvArgs {
  Segments g;
  const void* x;
  const void* w;     // [channels, K]
  const void* bias;  // [channels] or NULL
  void* state;       // [R, K - 1, channels]
  void* out;
  int64_t ldx, ldo;
  int32_t channels, act, tokens, runs, blocks;  // tokens: TT; blocks: CTAs across the channels
};

constexpr int kConvThreads = 128;
constexpr int kConvMaxRun = 16;
constexpr int kConvCh = 4;  // channels of a thread

// One thread's 4 channels: weights and the sum over the K taps.
template <typename T, int K>
struct ConvLane {
  struct Four {
    f32x2 v[2];  // channel pairs
  };
  f32x2 w[K][2], b[2];
  int32_t act;

  __device__ __forceinline__ void load(const ConvArgs& p, int32_t c) {
    act = p.act;
    float wf[4 * K];  // wf[i * K + k]: channel i, tap k (memory order)
#pragma unroll
    for (int k = 0; k < K; ++k)
      unpack4<T>(reinterpret_cast<const uint2*>(static_cast<const T*>(p.w) +
                                                static_cast<int64_t>(c) * K)[k], wf + 4 * k);
    float bf[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias)
      unpack4<T>(*reinterpret_cast<const uint2*>(static_cast<const T*>(p.bias) + c), bf);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      b[e] = pack2(bf[2 * e], bf[2 * e + 1]);
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][e] = pack2(wf[2 * e * K + k], wf[(2 * e + 1) * K + k]);
    }
  }
  static __device__ __forceinline__ Four widen(const uint2& raw) {
    float f[4];
    unpack4<T>(raw, f);
    return Four{{pack2(f[0], f[1]), pack2(f[2], f[3])}};
  }
  // the output of the token whose K inputs are v[0] .. v[K - 1]
  __device__ __forceinline__ uint2 token(const Four* v) const {
    float y[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f32x2 a = b[e];
#pragma unroll
      for (int k = 0; k < K; ++k) a = fma2(w[k][e], v[k].v[e], a);
      unpack2(a, y[2 * e], y[2 * e + 1]);
    }
    if (act) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = silu(y[e]);
    }
    return pack4<T>(y);
  }
};

// kPack whole segments of at most kShortTokens tokens, from s on.
constexpr int kPack = 2;
template <typename T, int K>
__device__ __forceinline__ void conv_short(const ConvArgs& p, int32_t s, int32_t c) {
  using L = ConvLane<T, K>;
  L lane;
  lane.load(p, c);
  Segment g[kPack];
#pragma unroll
  for (int e = 0; e < kPack; ++e) {
    g[e] = {0, 0, -1, 0};
    if (s + e < p.g.S) g[e] = read_segment(p.g, s + e);
  }
  const int64_t ldx = p.ldx / 4, ldo = p.ldo / 4, lds = p.channels / 4;
  const uint2* X[kPack];
  uint2* kept[kPack];
  uint2 raw[kPack][K];  // the kept inputs and the first token's
#pragma unroll
  for (int e = 0; e < kPack; ++e) {
    const int32_t len = g[e].q1 - g[e].q0;
    if (len <= 0 || len > kShortTokens) g[e].id = -1;
    if (g[e].id < 0) continue;
    X[e] = reinterpret_cast<const uint2*>(static_cast<const T*>(p.x) + g[e].q0 * p.ldx + c);
    kept[e] = reinterpret_cast<uint2*>(static_cast<T*>(p.state) +
                                       static_cast<int64_t>(g[e].id) * (K - 1) * p.channels + c);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) raw[e][k] = g[e].old ? kept[e][k * lds] : make_uint2(0u, 0u);
    raw[e][K - 1] = X[e][0];
  }
#pragma unroll
  for (int e = 0; e < kPack; ++e) {
    if (g[e].id < 0) continue;
    const int32_t len = g[e].q1 - g[e].q0;
    uint2* O = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + g[e].q0 * p.ldo + c);
    uint2 more[kShortTokens - 1];
#pragma unroll
    for (int i = 1; i < kShortTokens; ++i)
      if (i < len) more[i - 1] = X[e][i * ldx];
    typename L::Four win[K];
#pragma unroll
    for (int k = 0; k < K; ++k) win[k] = L::widen(raw[e][k]);
    O[0] = lane.token(win);
#pragma unroll
    for (int i = 1; i < kShortTokens; ++i) {
      if (i >= len) break;
#pragma unroll
      for (int k = 0; k + 1 < K; ++k) {
        win[k] = win[k + 1];
        raw[e][k] = raw[e][k + 1];
      }
      raw[e][K - 1] = more[i - 1];
      win[K - 1] = L::widen(more[i - 1]);
      O[i * ldo] = lane.token(win);
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) kept[e][k * lds] = raw[e][k + 1];
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads, 8) mixed_conv_kernel(const ConvArgs p) {
  if (blockIdx.x == 0) {
    check_segments(p.g);
    return;
  }
  const int32_t c = ((blockIdx.x - 1) % p.blocks * kConvThreads + threadIdx.x) * kConvCh;
  const int32_t tile = (blockIdx.x - 1) / p.blocks;
  // the runs first: they take longest (2048 tokens and 64 decodes of 8192
  // channels 17.3 us, behind the decodes 18.0)
  if (tile >= p.runs) {
    if (c < p.channels) conv_short<T, K>(p, (tile - p.runs) * kPack, c);
    return;
  }
  using L = ConvLane<T, K>;
  constexpr int kBatch = 4;  // inputs requested together
  __shared__ Segment info[kConvMaxRun + K];
  __shared__ int32_t first;
  const int32_t t0 = tile * p.tokens;
  const int32_t run = min(p.tokens, p.g.T - t0);
  const int32_t most = min(p.tokens + K - 2, p.g.T - t0);  // with a head that goes on
  // the weights and the first inputs are on their way while the segments are looked up
  const int32_t cc = min(c, p.channels - kConvCh);
  const uint2* X = reinterpret_cast<const uint2*>(static_cast<const T*>(p.x) + cc);
  uint2* O = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + cc);
  const int64_t ldx = p.ldx / 4, ldo = p.ldo / 4, lds = p.channels / 4;
  L lane;
  lane.load(p, cc);
  uint2 raw[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (i < run) raw[i] = X[(t0 + i) * ldx];

  // segments before the first token: those that end at or before it
  const int32_t t = t0 + threadIdx.x;
  if (threadIdx.x == 0) first = 0;
  __syncthreads();
  int32_t n = 0;
  for (int32_t s = threadIdx.x; s < p.g.S; s += kConvThreads) n += p.g.cu[s + 1] <= t0;
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&first, n);
  __syncthreads();
  if (threadIdx.x < most) {
    int32_t lo = first, hi = p.g.S;  // first segment that ends behind t
    Segment mine = {0, 0, -1, 0};
    if (lo < hi) mine = read_segment(p.g, lo);
    if (lo < hi && mine.q1 <= t) {
      ++lo;
      while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (p.g.cu[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
      }
      if (lo < p.g.S) mine = read_segment(p.g, lo);
    }
    // not a short segment's token; a segment's first K - 1 tokens belong to the
    // run that its first token is in
    const int32_t off = t - mine.q0;
    if (off < 0 || t >= mine.q1 || mine.q1 - mine.q0 <= kShortTokens ||
        !(off < K - 1 ? mine.q0 >= t0 && mine.q0 < t0 + run : t < t0 + run))
      mine.id = -1;
    info[threadIdx.x] = mine;
  }
  __syncthreads();
  if (c >= p.channels) return;

  const Segment head = info[0];
  if (run == p.tokens && run % kBatch == 0 && head.id >= 0 && t0 - head.q0 >= K - 1 &&
      t0 + run <= head.q1) {
    // the whole run lies inside one segment, behind its first tokens
    const uint2* from = X + t0 * ldx;
    uint2* to = O + t0 * ldo;
    typename L::Four v[K - 1 + kBatch];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) v[k] = L::widen(from[(k - K + 1) * ldx]);
    for (int i0 = 0; i0 < run; i0 += kBatch) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[K - 1 + i] = L::widen(raw[i]);
      if (i0 + kBatch < run) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) raw[i] = from[(kBatch + i) * ldx];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) to[i * ldo] = lane.token(v + i);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) v[k] = v[kBatch + k];
      from += kBatch * ldx;
      to += kBatch * ldo;
    }
    return;
  }
  typename L::Four win[K];  // the K - 1 inputs before the next token, then its own
  bool have = false;        // they are there
  for (int32_t i0 = 0; i0 < most; i0 += kBatch) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < most && (i0 > 0 || i >= run) && info[i0 + i].id >= 0) raw[i] = X[(t0 + i0 + i) * ldx];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int32_t at = i0 + i;
      if (at >= most) break;
      const Segment s = info[at];
      const int32_t tok = t0 + at, off = tok - s.q0;
      if (s.id < 0) {
        have = false;
        continue;
      }
      if (off == 0) {
        uint2* kept = reinterpret_cast<uint2*>(static_cast<T*>(p.state) +
                                               static_cast<int64_t>(s.id) * (K - 1) * p.channels + c);
#pragma unroll
        for (int k = 0; k < K - 1; ++k) win[k] = L::widen(s.old ? kept[k * lds] : make_uint2(0u, 0u));
        // the kept inputs of the next step (a segment has more than K - 1 tokens here)
#pragma unroll
        for (int k = 0; k < K - 1; ++k) kept[k * lds] = X[(s.q1 - (K - 1) + k) * ldx];
      } else if (!have) {
        // behind a first token of another segment's: a prefix sum that decreases
        // (reported); the inputs before this one may lie outside the stream
        if (off < K - 1) continue;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) win[k] = L::widen(X[(tok - (K - 1) + k) * ldx]);
      }
      have = true;
      win[K - 1] = L::widen(raw[i]);
      O[tok * ldo] = lane.token(win);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) win[k] = win[k + 1];
    }
  }
}

template <typename T, int K>
int conv_launch(const ConvArgs& a, int64_t grid, cudaStream_t st) {
  mixed_conv_kernel<T, K><<<static_cast<unsigned>(grid), kConvThreads, 0, st>>>(a);
  return static_cast<int>(cudaGetLastError());
}
template <typename T>
int conv_width(const ConvArgs& a, int K, int64_t grid, cudaStream_t st) {
  if (K == 2) return conv_launch<T, 2>(a, grid, st);
  if (K == 3) return conv_launch<T, 3>(a, grid, st);
  return conv_launch<T, 4>(a, grid, st);
}

// --------------------------------------------------------------------- scan
// Per channel c and state n, along a segment's tokens:
//   d = softplus(dt + dt_bias),  h = exp(d A[c, n]) h + d x B[n],
//   y = sum_n C[n] h[c, n] + D[c] x,  out = y silu(z).
// State and sums are fp32.  exp(d A) is ex2.approx of d (A log2 e): the 2 ulp of
// the instruction and three roundings of its argument, (4 + 3 |d A|) 2^-24 of it,
// beside the error of d; the recurrence multiplies by it once a token.
//
// Least traffic: x, dt, z read and out written once (8 bytes per token and
// channel in 16 bits) and the states once.  Segments of a few tokens (decodes)
// are bound by their states' traffic, long ones by one ex2 per token, channel
// and state (32 a clock and SM: 16 states take longer than the HBM traffic)
// and by the issue slots of the recurrence.  They run in two kernels.
struct ScanArgs {
  Segments g;
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* dt_bias;
  float* state;
  void* out;
  int64_t ldx, lddt, ldz, ldb, ldc, ldo;
  int32_t channels, per_group, softplus;
  int32_t blocks;     // warps across the channels
  int32_t split;      // warps the short segments are dealt to
  int32_t short_max;  // segments of at most this many tokens are the short kernel's
  int32_t piece;      // longer segments are cut into pieces of at most so many tokens (0: not)
  int32_t slots;      // room for pieces that another follows
  int32_t* counter;   // in the workspace, as the sums and end states behind it
  float* carries;
};

// max(v, 0) + log1p(exp(-|v|)), two values at a time, to a few ulp also where
// it is small (steps of 0.001 and less).  exp(-u) = 2^(hi - lo): hi the rounded
// product -u log2 e, lo what the rounding lost.  log1p(e) = e P(e) on [0, 1], P
// of degree 8 from a Remez exchange on the relative error (3e-8); Horner's
// roundings leave 3 x 2^-24 in all.
__device__ __forceinline__ void softplus2(float& v0, float& v1) {
  // u = |v|, at most 128: exp(-128) is 0 in fp32, and of an infinite product
  // nothing finite is lost
  const f32x2 u = pack2(least(fabsf(v0), 128.f), least(fabsf(v1), 128.f));
  const f32x2 hi = mul2(u, pack2(-kLog2e, -kLog2e));
  // log2 e - float(log2 e) = 1.925963e-8
  const f32x2 lo = fma2(u, pack2(1.925963033e-8f, 1.925963033e-8f), fma2(u, pack2(kLog2e, kLog2e), hi));
  f32x2 e = ex2x2(hi);
  e = fma2(e, mul2(lo, pack2(-kLn2, -kLn2)), e);
  f32x2 q = pack2(5.2326940931379795e-3f, 5.2326940931379795e-3f);
  q = fma2(q, e, pack2(-2.950523979961872e-2f, -2.950523979961872e-2f));
  q = fma2(q, e, pack2(7.822595536708832e-2f, 7.822595536708832e-2f));
  q = fma2(q, e, pack2(-1.3663245737552643e-1f, -1.3663245737552643e-1f));
  q = fma2(q, e, pack2(1.9106006622314453e-1f, 1.9106006622314453e-1f));
  q = fma2(q, e, pack2(-2.484298199415207e-1f, -2.484298199415207e-1f));
  q = fma2(q, e, pack2(3.331909775733948e-1f, 3.331909775733948e-1f));
  q = fma2(q, e, pack2(-4.999949336051941e-1f, -4.999949336051941e-1f));
  q = fma2(q, e, pack2(9.999999403953552e-1f, 9.999999403953552e-1f));
  float p0, p1;
  unpack2(mul2(q, e), p0, p1);
  v0 = fmaxf(v0, 0.f) + p0;
  v1 = fmaxf(v1, 0.f) + p1;
}

// ------------------------------------------------- scan of short segments
// A warp takes 16 (N = 16) channels and runs over its share of the segments: 4
// states of 2 channels a lane, so a request's state is two coalesced 16-byte
// accesses a lane.  A decode is one register-only step between the state's load
// and its store.  The bound is the states' HBM traffic (8 N bytes per channel
// and segment against 8), so what counts is bytes in flight and few
// instructions: the metadata of 32 segments come in one load each, the states
// and inputs of the next segments in asynchronous copies to the warp's ring in
// shared memory, and a second channel halves what a segment costs beside its
// arithmetic (with one, 225 instructions a warp and segment kept the issue slots
// 80% busy).  256 decodes of 8192 channels and 16 states: 48.6 us, 5.9 TB/s; one
// channel a lane 61 us.
//
// A call with at most as many tokens as segments has no other launch, and a padded
// step of it may hold a long segment.  The tokens behind a segment's first come in
// asynchronous copies as well, up to four ahead, over the state that was read (900
// tokens and 100 decodes of 8192 channels: 370 us, loaded one by one 914; with one
// row of tokens more, through the long segments' launches, 138).
template <typename T>
__device__ __forceinline__ float scalar(const T* p) {
  if constexpr (std::is_same<T, __half>::value) return __half2float(*p);
  else return __bfloat162float(*p);
}
// 4, 8 or 16 bytes global -> shared without a register in between
template <int n>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(n) : "memory");
}

constexpr int kShortThreads = 128;
constexpr int kAhead = 4;  // slots of the ring

template <int N>
struct ShortCfg {
  static constexpr int LPC = N / 4;                          // lanes of a channel
  static constexpr int kHalf = 32 / LPC;                     // a lane's channels are c and c + kHalf
  static constexpr int CPW = 2 * kHalf;                      // channels of a warp
  static constexpr int kXBytes = CPW * 2;                    // of x, dt, z each
  static constexpr int kXPiece = kXBytes < 16 ? kXBytes : 16;
  static constexpr int kXPieces = kXBytes / kXPiece;
  static constexpr int kBPieces = N * 2 / 16;                // of B and C each
  static constexpr int kX = 1024;                            // offsets in a slot: state first
  static constexpr int kB = kX + (3 * kXBytes + 15) / 16 * 16;
  static constexpr int kSlot = kB + 2 * N * 2;
  static constexpr int kInputs = kSlot - kX;                 // bytes of a token beside the state
  static constexpr int kTokens = 1024 / kInputs < 4 ? 1024 / kInputs : 4;  // that fit over a state
};

template <typename T, int N>
__global__ void __launch_bounds__(kShortThreads) scan_short_kernel(const ScanArgs p) {
  // nothing here depends on the long segments' launches, which this one may run
  // beside; it ends behind them
  if (blockIdx.x == 0) {
    check_segments(p.g);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  using C = ShortCfg<N>;
  constexpr int LPC = C::LPC, CPW = C::CPW;
  __shared__ __align__(16) unsigned char rings[kShortThreads / 32][kAhead][C::kSlot];
  const int lane = threadIdx.x & 31, sub = lane % LPC, cl = lane / LPC;
  unsigned char(*ring)[C::kSlot] = rings[threadIdx.x >> 5];
  const int32_t wid = (blockIdx.x - 1) * (kShortThreads / 32) + (threadIdx.x >> 5);
  const int32_t c0 = wid % p.blocks * CPW;  // blocks: warps across the channels
  const int32_t first = wid / p.blocks;
  if (first >= p.split) return;
  const int32_t gn = c0 / p.per_group * N;
  bool live[2];
  int32_t cc[2];
  float a[2][4], bias[2], skip[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int32_t c = c0 + cl + e * C::kHalf;
    live[e] = c < p.channels;
    cc[e] = live[e] ? c : p.channels - 1;  // idle lanes shadow the last channel
    const float4 v = *reinterpret_cast<const float4*>(p.A + static_cast<int64_t>(cc[e]) * N + 4 * sub);
    a[e][0] = v.x * kLog2e, a[e][1] = v.y * kLog2e, a[e][2] = v.z * kLog2e, a[e][3] = v.w * kLog2e;
    bias[e] = p.dt_bias ? p.dt_bias[cc[e]] : 0.f;
    skip[e] = p.D ? p.D[cc[e]] : 0.f;
  }

  // this lane's part of a segment's inputs beside the state: a piece of x, dt, z
  // (what 0 .. 2) or of B, C (3, 4), or nothing (-1)
  int what = -1, to = 0;
  const T* src = nullptr;
  int64_t ld = 0;
  if (lane < 3 * C::kXPieces) {
    const int k = lane / C::kXPieces, piece = lane % C::kXPieces;
    const int32_t ch = c0 + piece * (C::kXPiece / 2);
    const void* base = k == 0 ? p.x : k == 1 ? p.dt : p.z;
    if (base && ch < p.channels) {
      what = k;
      src = static_cast<const T*>(base) + ch;
      ld = k == 0 ? p.ldx : k == 1 ? p.lddt : p.ldz;
      to = C::kX + k * C::kXBytes + piece * C::kXPiece;
    }
  } else if (lane < 3 * C::kXPieces + 2 * C::kBPieces) {
    const int k = (lane - 3 * C::kXPieces) / C::kBPieces, piece = (lane - 3 * C::kXPieces) % C::kBPieces;
    what = 3 + k;
    src = static_cast<const T*>(k ? p.C : p.B) + gn + 8 * piece;
    ld = k ? p.ldc : p.ldb;
    to = C::kB + k * 2 * N + 16 * piece;
  }
  const int64_t row = static_cast<int64_t>(p.channels) * N;
  float* const state = p.state + static_cast<int64_t>(c0 + cl) * N + 4 * sub;
  auto request = [&](int32_t q0, int32_t id, int32_t old, int slot) {
    if (id >= 0) {
      if (old) {
        const float* from = state + id * row;
        if (live[0]) copy_async<16>(ring[slot] + 16 * lane, from);
        if (live[1]) copy_async<16>(ring[slot] + 512 + 16 * lane, from + C::kHalf * N);
      }
      if (what >= 3) copy_async<16>(ring[slot] + to, src + q0 * ld);
      else if (what >= 0) copy_async<C::kXPiece>(ring[slot] + to, src + q0 * ld);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // segments first + k split, k = k0 .. k0 + 31 in the lanes' registers
  for (int32_t s0 = first; s0 < p.g.S; s0 += 32 * p.split) {
    Segment m = {0, 0, -1, 0};
    if (s0 + static_cast<int64_t>(lane) * p.split < p.g.S) m = read_segment(p.g, s0 + lane * p.split);
    if (m.q1 <= m.q0 || m.q1 - m.q0 > p.short_max) m.id = -1;
    // the segments to do, moved to the front
    uint32_t todo = __ballot_sync(0xffffffffu, m.id >= 0);
    const int n = __popc(todo);
    const int from = __fns(todo, 0, lane + 1) & 31;
    m.q0 = __shfl_sync(0xffffffffu, m.q0, from);
    m.q1 = __shfl_sync(0xffffffffu, m.q1, from);
    m.id = __shfl_sync(0xffffffffu, m.id, from);
    m.old = __shfl_sync(0xffffffffu, m.old, from);
    if (lane >= n) m.id = -1;
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i)
      request(__shfl_sync(0xffffffffu, m.q0, i), __shfl_sync(0xffffffffu, m.id, i),
              __shfl_sync(0xffffffffu, m.old, i), i);
    for (int i = 0; i < n; ++i) {
      const int ahead = i + kAhead - 1;
      int32_t id = __shfl_sync(0xffffffffu, m.id, ahead & 31);
      if (ahead >= 32) id = -1;
      request(__shfl_sync(0xffffffffu, m.q0, ahead & 31), id, __shfl_sync(0xffffffffu, m.old, ahead & 31),
              ahead % kAhead);
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      __syncwarp();
      const unsigned char* slot = ring[i % kAhead];
      const int32_t q0 = __shfl_sync(0xffffffffu, m.q0, i), q1 = __shfl_sync(0xffffffffu, m.q1, i);
      const int32_t old = __shfl_sync(0xffffffffu, m.old, i);
      id = __shfl_sync(0xffffffffu, m.id, i);
      float h[2][4], x[2], d[2], z[2];
      uint2 b, q;
      auto inputs = [&](const unsigned char* at) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const T* xs = reinterpret_cast<const T*>(at) + cl + e * C::kHalf;
          x[e] = scalar<T>(xs);
          d[e] = scalar<T>(xs + CPW);
          z[e] = p.z ? scalar<T>(xs + 2 * CPW) : 0.f;
        }
        b = *reinterpret_cast<const uint2*>(at + C::kB - C::kX + 8 * sub);
        q = *reinterpret_cast<const uint2*>(at + C::kB - C::kX + 2 * N + 8 * sub);
      };
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (old) v = *reinterpret_cast<const float4*>(slot + 512 * e + 16 * lane);
        h[e][0] = v.x, h[e][1] = v.y, h[e][2] = v.z, h[e][3] = v.w;
      }
      inputs(slot + C::kX);
      // the tokens behind the first, a few ahead, over the state that was read
      auto token = [&](int32_t t) {
        unsigned char* at = ring[i % kAhead] + (t - q0) % C::kTokens * C::kInputs + to - C::kX;
        if (t < q1) {
          if (what >= 3) copy_async<16>(at, src + t * ld);
          else if (what >= 0) copy_async<C::kXPiece>(at, src + t * ld);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if (q1 - q0 > 1) {
        __syncwarp();
#pragma unroll
        for (int k = 1; k <= C::kTokens; ++k) token(q0 + k);
      }
      for (int32_t t = q0;;) {
        float bb[4], qq[4], y[2];
        unpack4<T>(b, bb);
        unpack4<T>(q, qq);
        float d0 = d[0] + bias[0], d1 = d[1] + bias[1];
        if (p.softplus) softplus2(d0, d1);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float dd = e ? d1 : d0, dx = dd * x[e];
          y[e] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            h[e][k] = fmaf(ex2(dd * a[e][k]), h[e][k], dx * bb[k]);
            y[e] = fmaf(qq[k], h[e][k], y[e]);
          }
        }
        // the first exchange leaves a lane with one of the two channels
        float s;
        {
          const bool up = lane & 1;
          const float give = up ? y[0] : y[1], keep = up ? y[1] : y[0];
          s = keep + __shfl_xor_sync(0xffffffffu, give, 1);
        }
#pragma unroll
        for (int o = 2; o < LPC; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (sub < 2) {
          const int e = sub;
          s = fmaf(e ? skip[1] : skip[0], e ? x[1] : x[0], s);
          if (p.z) s *= silu(e ? z[1] : z[0]);
          if (e ? live[1] : live[0])
            static_cast<T*>(p.out)[t * p.ldo + (e ? cc[1] : cc[0])] = static_cast<T>(s);
        }
        if (++t >= q1) break;
        asm volatile("cp.async.wait_group %0;" ::"n"(C::kTokens - 1) : "memory");
        __syncwarp();
        inputs(slot + (t - q0) % C::kTokens * C::kInputs);
        __syncwarp();
        token(t + C::kTokens);
      }
      float* to_state = state + id * row;
      if (live[0]) *reinterpret_cast<float4*>(to_state) = make_float4(h[0][0], h[0][1], h[0][2], h[0][3]);
      if (live[1])
        *reinterpret_cast<float4*>(to_state + C::kHalf * N) = make_float4(h[1][0], h[1][1], h[1][2], h[1][3]);
      __syncwarp();  // the slot is read before it is requested again
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // the empty tail
    __syncwarp();
  }
}

// -------------------------------------------------- scan of long segments
// A lane holds up to 16 states of 2 neighbouring channels (N = 16: a warp has 64
// channels, and nothing crosses its lanes), so a token's d, d x, y and output
// stay in its registers, and shared memory gives it only B and C.  That is what
// the layout is for: shared memory returns 128 bytes a clock, also for a
// broadcast, and with fewer states times channels a lane the B and C loads
// alone (32 to 40 clocks an SM for 32 channels of a token) outweigh the
// arithmetic.  That is 110 instructions for 32 channels of a token and 16
// states, 19 of them ex2 or reciprocals, some 40 packed pairs that take two
// issue slots each: 184 clocks a sub-partition (1.24 M such groups, 12 x 340 tokens
// of 9728 channels: 192 us).  With 3 instructions less in the gate it was 178,
// whether 8, 12 or 16 warps an SM ran, with scalar products in place of the pairs or
// not; a lane of one channel needed 153 instructions and 221 clocks.  The next token's softplus stands beside the
// recurrence, 32 independent chains of it.
//
// Tiles of 16 tokens of x, dt, z, B and C come in asynchronous copies to the
// warp's own ring in shared memory, two tiles deep; there is no barrier but the
// warp's.
//
// Tasks are (piece of a segment, 64 channels).  A segment of more than `piece`
// tokens is cut, so that a lone chunk fills the GPU and the longest prompt of a
// batch does not outlast the others.  The first launch takes the whole segments
// and each cut one's piece 0, whose start is known, and runs the pieces between
// the first and the last from a zero state, without C and y: that leaves the
// state e they end with and the sum s of their d.  A small launch then carries
// piece 0's end over them, e_j <- exp(s_j A) e_{j-1} + e_j, and the last runs
// pieces 1 and up from those states.  Only pieces in between run one and a half
// times, and a request's state is read in the first launch and written in the
// last.
constexpr int long_warps(int N) { return N < 64 ? 12 : 8; }  // of a CTA, one CTA an SM
constexpr int kTile = 16;
constexpr int64_t kCutTenths = 8;   // a piece's tokens in tenths of a warp slot's share
constexpr int kUncut = 4 * kTile;  // tokens

template <int N>
struct LongCfg {
  static constexpr int NS = N < 16 ? N : 16;  // states of a lane
  static constexpr int LPC = N / NS;          // lanes of a channel
  static constexpr int CPW = 64 / LPC;        // channels of a warp
  static constexpr int kRow = CPW * 2;        // bytes of a token's x, dt or z
  static constexpr int kBRow = N * 2;         // of its B or C
  static constexpr int kRaw = kTile * (3 * kRow + 2 * kBRow);  // a stage of the ring
  static constexpr int kWarpBytes = 2 * kRaw + 2 * kTile * N * 4;
  static constexpr int kWarps = long_warps(N);
  static constexpr int kSmem = kWarps * kWarpBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
};

template <typename T, int N>
struct LongScan {
  using C = LongCfg<N>;
  const ScanArgs& p;
  unsigned char* ring;
  float* bc;          // [2][kTile][N] fp32
  int lane, cl, sub;  // cl: first of the lane's two channels in the warp's
  int32_t cb, end, group;  // the warp's channels (up to the group's end)
  float bias[2], skip[2];
  f32x2 a[2][C::NS / 2], h[2][C::NS / 2];
  float sum[2];

  __device__ __forceinline__ void block(int32_t b) {
    const int32_t per = (p.per_group + C::CPW - 1) / C::CPW;  // blocks of a group
    group = b / per;
    end = (group + 1) * p.per_group;
    cb = group * p.per_group + (b - group * per) * C::CPW;
  }
  __device__ __forceinline__ void weights() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t c = min(cb + cl + e, p.channels - 1);
#pragma unroll
      for (int n = 0; n < C::NS / 4; ++n) {
        const float4 v = *reinterpret_cast<const float4*>(p.A + c * N + sub * C::NS + 4 * n);
        a[e][2 * n] = pack2(v.x * kLog2e, v.y * kLog2e);
        a[e][2 * n + 1] = pack2(v.z * kLog2e, v.w * kLog2e);
      }
      bias[e] = p.dt_bias ? p.dt_bias[c] : 0.f;
      skip[e] = p.D ? p.D[c] : 0.f;
    }
  }
  // Rows of `bytes` bytes of tokens t0 .. t0 + nt - 1 into a ring stage.
  template <int kBytes>
  __device__ __forceinline__ void copy_rows(unsigned char* to, const T* from, int64_t ld, int nt,
                                            int32_t limit) {
    constexpr int kPieces = kBytes / 16, kAll = kTile * kPieces;
#pragma unroll
    for (int i = 0; i < (kAll + 31) / 32; ++i) {
      const int k = lane + 32 * i, row = k / kPieces, piece = k % kPieces;
      if ((kAll % 32 == 0 || k < kAll) && row < nt && piece * 8 < limit)
        copy_async<16>(to + 16 * k, from + row * ld + piece * 8);
    }
  }
  template <bool kAll>
  __device__ __forceinline__ void request(int32_t t0, int32_t t1, int stage) {
    const int nt = min(kTile, t1 - t0);
    unsigned char* to = ring + stage * C::kRaw;
    if (nt > 0) {
      const int64_t t = t0;
      const int32_t limit = end - cb;  // channels come in eights
      copy_rows<C::kRow>(to, static_cast<const T*>(p.x) + t * p.ldx + cb, p.ldx, nt, limit);
      copy_rows<C::kRow>(to + kTile * C::kRow, static_cast<const T*>(p.dt) + t * p.lddt + cb, p.lddt, nt, limit);
      if (kAll && p.z)
        copy_rows<C::kRow>(to + 2 * kTile * C::kRow, static_cast<const T*>(p.z) + t * p.ldz + cb, p.ldz, nt,
                           limit);
      unsigned char* tb = to + 3 * kTile * C::kRow;
      copy_rows<C::kBRow>(tb, static_cast<const T*>(p.B) + t * p.ldb + group * N, p.ldb, nt, N);
      if (kAll)
        copy_rows<C::kBRow>(tb + kTile * C::kBRow, static_cast<const T*>(p.C) + t * p.ldc + group * N, p.ldc,
                            nt, N);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ static void pair(const unsigned char* at, float& u, float& v) {
    float f[4];
    unpack4<T>(make_uint2(*reinterpret_cast<const uint32_t*>(at), 0u), f);
    u = f[0];
    v = f[1];
  }
  // (d, d x) of the lane's channels at a token of the stage
  struct Token {
    float d[2], x[2];
  };
  __device__ __forceinline__ Token token(const unsigned char* raw, int r) const {
    Token k;
    pair(raw + r * C::kRow + 2 * cl, k.x[0], k.x[1]);
    pair(raw + kTile * C::kRow + r * C::kRow + 2 * cl, k.d[0], k.d[1]);
    k.d[0] += bias[0];
    k.d[1] += bias[1];
    if (p.softplus) softplus2(k.d[0], k.d[1]);
    return k;
  }
  // Tokens [t0, t1), whose first tile is requested, from the state in h.  kAll
  // false: only the state and the sums of d.
  template <bool kAll>
  __device__ __forceinline__ void run(int32_t t0, int32_t t1) {
    int stage = 0;
    for (; t0 < t1; t0 += kTile, stage ^= 1) {
      __syncwarp();  // the stage before this one is done with
      request<kAll>(t0 + kTile, t1, stage ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      const int nt = min(kTile, t1 - t0);
      const unsigned char* raw = ring + stage * C::kRaw;
      // B and C as fp32 (what stands behind the last token is not used)
      constexpr int kVecs = 2 * kTile * N / 8;
#pragma unroll
      for (int i = 0; i < (kVecs + 31) / 32; ++i) {
        const int k = lane + 32 * i;
        if (k >= (kAll ? kVecs : kVecs / 2)) continue;
        float f[8];
        unpack8<T>(*reinterpret_cast<const uint4*>(raw + 3 * kTile * C::kRow + 16 * k), f);
        float4* to = reinterpret_cast<float4*>(bc + 8 * k);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
      __syncwarp();
      T* out = static_cast<T*>(p.out) + t0 * p.ldo + cb + cl;
      const ulonglong2* __restrict__ Bt = reinterpret_cast<const ulonglong2*>(bc + sub * C::NS);
      const ulonglong2* __restrict__ Ct = Bt + kTile * N / 4;
      Token cur = token(raw, 0);
#pragma unroll 2
      for (int r = 0; r < nt; ++r) {
        const Token nxt = token(raw, min(r + 1, nt - 1));
        float z0 = 0.f, z1 = 0.f;
        if (kAll && p.z) pair(raw + 2 * kTile * C::kRow + r * C::kRow + 2 * cl, z0, z1);
        f32x2 d[2], dx[2], y[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = cur.d[e] * cur.x[e];
          d[e] = pack2(cur.d[e], cur.d[e]);
          dx[e] = pack2(v, v);
          if (!kAll) sum[e] += cur.d[e];
        }
#pragma unroll
        for (int n = 0; n < C::NS / 4; ++n) {
          const ulonglong2 b = Bt[r * (N / 4) + n];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            h[e][2 * n] = fma2(ex2x2(mul2(d[e], a[e][2 * n])), h[e][2 * n], mul2(dx[e], b.x));
            h[e][2 * n + 1] = fma2(ex2x2(mul2(d[e], a[e][2 * n + 1])), h[e][2 * n + 1], mul2(dx[e], b.y));
          }
          if (kAll) {
            const ulonglong2 q = Ct[r * (N / 4) + n];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[e] = n ? fma2(h[e][2 * n], q.x, y[e]) : mul2(h[e][0], q.x);
              y[e] = fma2(h[e][2 * n + 1], q.y, y[e]);
            }
          }
        }
        if (kAll) {
          float s[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float u, v;
            unpack2(y[e], u, v);
            s[e] = u + v;
          }
          if constexpr (C::LPC > 1) {
#pragma unroll
            for (int o = 1; o < C::LPC; o <<= 1)
#pragma unroll
              for (int e = 0; e < 2; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
          }
          s[0] = fmaf(skip[0], cur.x[0], s[0]);
          s[1] = fmaf(skip[1], cur.x[1], s[1]);
          if (p.z) {
            s[0] *= silu(z0);
            s[1] *= silu(z1);
          }
          if (sub == 0 && cb + cl < end) {
            const float f[4] = {s[0], s[1], 0.f, 0.f};
            *reinterpret_cast<uint32_t*>(out + r * p.ldo) = pack4<T>(f).x;
          }
        }
        cur = nxt;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();  // the ring is done with
  }
  // h <-> memory [channels, N] at `base`
  __device__ __forceinline__ void read(const float* base) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const ulonglong2* at = reinterpret_cast<const ulonglong2*>(
          base + static_cast<int64_t>(min(cb + cl + e, p.channels - 1)) * N + sub * C::NS);
#pragma unroll
      for (int n = 0; n < C::NS / 4; ++n) {
        const ulonglong2 v = at[n];
        h[e][2 * n] = v.x;
        h[e][2 * n + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void write(float* base) const {
    if (cb + cl >= end) return;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ulonglong2* at =
          reinterpret_cast<ulonglong2*>(base + static_cast<int64_t>(cb + cl + e) * N + sub * C::NS);
#pragma unroll
      for (int n = 0; n < C::NS / 4; ++n) at[n] = make_ulonglong2(h[e][2 * n], h[e][2 * n + 1]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int n = 0; n < C::NS / 2; ++n) h[e][n] = 0;
  }
};

// Tokens of a piece: the shortest of a few lengths from p.piece on for which the
// first launch's tasks find a place together, or come in several rounds anyway;
// p.piece itself if there is none.  (A second round of a few tasks costs as much
// as a full one: 626 us instead of 488 for eight prompts of 8192 tokens in all.)
// The same in every warp.
__device__ __forceinline__ int32_t piece_of(const ScanArgs& p, int64_t places) {
  constexpr int kTries = 6;
  if (p.piece == 0) return 0;
  const int lane = threadIdx.x & 31;
  int32_t tasks[kTries] = {};
  for (int32_t s = lane; s < p.g.S; s += 32) {
    const Segment x = read_segment(p.g, s);
    const int32_t len = x.q1 - x.q0;
    if (x.id < 0 || len <= p.short_max) continue;
#pragma unroll
    for (int k = 0; k < kTries; ++k) {
      const int32_t piece = p.piece + p.piece / 8 * k;
      tasks[k] += max(1, (len + piece - 1) / piece - 1);
    }
  }
  int32_t piece = p.piece;
#pragma unroll
  for (int k = kTries - 1; k >= 0; --k) {
    const int64_t n = static_cast<int64_t>(__reduce_add_sync(0xffffffffu, tasks[k])) * p.blocks;
    if (n <= places || n > 4 * places) piece = p.piece + p.piece / 8 * k;
  }
  return piece;
}

// kFirst: whole segments, pieces 0, and what the pieces in between leave; else
// pieces 1 and up.  p.carries: sums [slots, channels] and end states [slots,
// channels, N] of the pieces that another follows; p.counter: what the second
// launch takes its tasks from (the first deals them in turn).
template <typename T, int N, bool kFirst>
__global__ void __launch_bounds__(32 * long_warps(N), 1) scan_long_kernel(const ScanArgs p) {
  using C = LongCfg<N>;
  extern __shared__ __align__(16) unsigned char smem[];
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char* mine = smem + warp * C::kWarpBytes;
  LongScan<T, N> w{p, mine, reinterpret_cast<float*>(mine + 2 * C::kRaw)};
  w.lane = lane;
  w.sub = lane % C::LPC;
  w.cl = lane / C::LPC * 2;
  float* const sums = p.carries;
  float* const ends = p.carries + static_cast<int64_t>(p.slots) * p.channels;
  const int64_t state = static_cast<int64_t>(p.channels) * N;
  if (kFirst && p.counter && blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;

  // dealt over the CTAs first: neighbouring tasks (pieces of one length) on
  // different SMs
  int32_t task = blockIdx.x + warp * gridDim.x;
  const int32_t piece = piece_of(p, static_cast<int64_t>(p.g.sms) * C::kWarps);
  // 32 segments from s0 on, in the lanes: pieces of each; tasks and slots before
  int32_t s0 = 0, base = 0, slot0 = 0;
  Segment m;
  int32_t k = 0, tasks = 0, incl = 0, slots_incl = 0;
  auto chunk = [&]() {
    m = {0, 0, -1, 0};
    if (s0 + lane < p.g.S) m = read_segment(p.g, s0 + lane);
    const int32_t len = m.q1 - m.q0;
    k = m.id < 0 || len <= p.short_max ? 0 : piece > 0 ? (len + piece - 1) / piece : 1;
    slots_incl = k > 1 ? k - 1 : 0;
    tasks = incl = kFirst && k == 1 ? 1 : slots_incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, incl, o), v = __shfl_up_sync(0xffffffffu, slots_incl, o);
      if (lane >= o) incl += u, slots_incl += v;
    }
  };
  chunk();
  if (!kFirst) asm volatile("griddepcontrol.wait;" ::: "memory");  // the carry is over
  while (true) {
    if (task < 0) return;  // past 2^31: overlapping segments (reported), see mixed_scan_fits
    const int32_t at = task / p.blocks;
    while (at >= base + __shfl_sync(0xffffffffu, incl, 31)) {
      base += __shfl_sync(0xffffffffu, incl, 31);
      slot0 += __shfl_sync(0xffffffffu, slots_incl, 31);
      s0 += 32;
      if (s0 >= p.g.S) return;
      chunk();
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, base + incl > at)) - 1;
    Segment s;
    s.q0 = __shfl_sync(0xffffffffu, m.q0, from);
    s.q1 = __shfl_sync(0xffffffffu, m.q1, from);
    s.id = __shfl_sync(0xffffffffu, m.id, from);
    s.old = __shfl_sync(0xffffffffu, m.old, from);
    const int32_t pieces = __shfl_sync(0xffffffffu, k, from);
    const int32_t i = at - (base + __shfl_sync(0xffffffffu, incl - tasks, from)) + (kFirst ? 0 : 1);
    const int32_t slot = slot0 + __shfl_sync(0xffffffffu, slots_incl, from) - (pieces - 1);  // of piece 0
    const int32_t len = s.q1 - s.q0;
    const int32_t size = ((len + pieces - 1) / pieces + kTile - 1) / kTile * kTile;
    const int32_t t0 = min(s.q1, s.q0 + i * size), t1 = min(s.q1, t0 + size);
    const int32_t now = task;
    if (kFirst) {
      task += gridDim.x * C::kWarps;
    } else {
      int32_t next = 0;
      if (lane == 0) next = atomicAdd(p.counter, 1);
      task = gridDim.x * C::kWarps + __shfl_sync(0xffffffffu, next, 0);
    }
    // overlapping segments (reported) could ask for more slots than there are
    if (pieces > 1 && slot + pieces - 1 > p.slots) continue;
    w.block(now % p.blocks);
    float* st = p.state + s.id * state;
    const bool carry = kFirst && i > 0;
    // the first tile is on its way while the weights and the start are read
    if (carry) w.template request<false>(t0, t1, 0);
    else w.template request<true>(t0, t1, 0);
    w.weights();
    if (carry) {
      w.clear();
      w.sum[0] = w.sum[1] = 0.f;
      w.template run<false>(t0, t1);
      if (w.sub == 0 && w.cb + w.cl < w.end)
        *reinterpret_cast<float2*>(sums + static_cast<int64_t>(slot + i) * p.channels + w.cb + w.cl) =
            make_float2(w.sum[0], w.sum[1]);
    } else {
      if (!kFirst) {
        w.read(ends + (slot + i - 1) * state);
      } else if (s.old) {
        w.read(st);
      } else {
        w.clear();
      }
      w.template run<true>(t0, t1);
    }
    w.write(i == pieces - 1 ? st : ends + (slot + i) * state);
  }
}

// h 2^t + v.  The factor of a whole piece can leave fp32 where the product does
// not (h = 0, or a small h that grew), so it is taken as the cube of 2^(t/3): at t/3
// = 126 every h but 0 has overflowed, below -126 nothing is left of any.
__device__ __forceinline__ float carried(float t, float h, float v) {
  const float f = ex2(least(t * (1.f / 3.f), 126.f));
  return fmaf(h * f * f, f, v);
}

// The end states of cut segments' pieces 1 .. (all but the last) from those they
// ended with from zero, in place.  A warp takes 128 states (four a lane) along
// every cut segment; the loads do not depend on each other.
constexpr int kCarryThreads = 128;
constexpr int kCarryLoads = 16;  // pieces whose loads are in flight together

template <int N>
__global__ void __launch_bounds__(kCarryThreads) scan_carry_kernel(const ScanArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t state = static_cast<int64_t>(p.channels) * N;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kCarryThreads + threadIdx.x) * 4;
  asm volatile("griddepcontrol.launch_dependents;");
  const bool live = at < state;
  const int32_t c = live ? static_cast<int32_t>(at / N) : 0;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) a = *reinterpret_cast<const float4*>(p.A + at);
  const float* sums = p.carries + c;
  float* ends = p.carries + static_cast<int64_t>(p.slots) * p.channels + (live ? at : 0);
  const int32_t piece = piece_of(p, static_cast<int64_t>(p.g.sms) * LongCfg<N>::kWarps);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the first launch is over
  int32_t slot0 = 0;
  for (int32_t s0 = 0; s0 < p.g.S; s0 += 32) {
    Segment m = {0, 0, -1, 0};
    if (s0 + lane < p.g.S) m = read_segment(p.g, s0 + lane);
    const int32_t len = m.q1 - m.q0;
    const int32_t own = m.id < 0 || len <= p.short_max ? 0 : (len + piece - 1) / piece - 1;
    int32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, own > 1); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int32_t n = __shfl_sync(0xffffffffu, own, from);
      const int32_t slot = slot0 + __shfl_sync(0xffffffffu, incl, from) - n;
      if (!live || slot + n > p.slots) continue;
      float4 h = *reinterpret_cast<const float4*>(ends + slot * state);
      for (int32_t j0 = 1; j0 < n; j0 += kCarryLoads) {
        float s[kCarryLoads];
        float4 v[kCarryLoads];
#pragma unroll
        for (int j = 0; j < kCarryLoads; ++j) {
          if (j0 + j >= n) break;
          // finite, so that A = 0 keeps its state (steps without softplus may be negative)
          s[j] = greatest(least(sums[static_cast<int64_t>(slot + j0 + j) * p.channels], 2e38f), -2e38f) * kLog2e;
          v[j] = *reinterpret_cast<const float4*>(ends + (slot + j0 + j) * state);
        }
#pragma unroll
        for (int j = 0; j < kCarryLoads; ++j) {
          if (j0 + j >= n) break;
          h.x = carried(s[j] * a.x, h.x, v[j].x);
          h.y = carried(s[j] * a.y, h.y, v[j].y);
          h.z = carried(s[j] * a.z, h.z, v[j].z);
          h.w = carried(s[j] * a.w, h.w, v[j].w);
          *reinterpret_cast<float4*>(ends + (slot + j0 + j) * state) = h;
        }
      }
    }
    slot0 += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// How a scan is cut: tokens of a piece, slots for the pieces that another follows.
struct ScanCut {
  int32_t piece, slots;
  size_t bytes;  // of workspace: the counter, the sums, the end states
};
// Warps of the long kernel across the channels; the segments that can be its.
int64_t long_blocks(const mcp_scan_desc& d) {
  const int ns = d.state_size < 16 ? d.state_size : 16, cpw = 64 / (d.state_size / ns);
  const int64_t per_group = d.channels / d.num_groups;
  return d.num_groups * ((per_group + cpw - 1) / cpw);
}
int64_t max_long(int32_t tokens, int32_t seqs) {
  const int32_t n = tokens / (kShortTokens + 1);
  return n < seqs ? n : seqs;
}
ScanCut scan_cut(const mcp_scan_desc& d, int sms) {
  // 0.8 of a warp slot's share of the work, in tokens (0.7 to 1 measured the same
  // on average, 0.5 and 1.2 5% to 10% longer), but not below 4 tiles: a piece's
  // start costs a tile or two.  2 tiles where 4 leave half of the slots empty (300
  // tokens of 4096 channels: 32 us instead of 47, 720 53 and 59; four segments of
  // 512 tokens and 2048 channels, which fill more, 75 instead of 66).
  const int64_t blocks = long_blocks(d), slots = static_cast<int64_t>(sms) * long_warps(d.state_size);
  const int64_t share = (d.total_tokens * blocks * kCutTenths + 10 * slots - 1) / (10 * slots);
  int64_t piece = (share + kTile - 1) / kTile * kTile;
  const bool few = d.total_tokens * blocks < slots / 2 * kUncut;
  if (piece < (few ? kUncut / 2 : kUncut)) piece = few ? kUncut / 2 : kUncut;
  ScanCut c = {0, 0, 0};
  if (d.total_tokens <= kUncut || d.total_tokens <= piece || d.total_tokens <= d.num_seqs) return c;
  c.piece = static_cast<int32_t>(piece);
  c.slots = static_cast<int32_t>(d.total_tokens / piece);
  c.bytes = 256 + static_cast<size_t>(c.slots) * d.channels * (d.state_size + 1) * sizeof(float);
  return c;
}

template <typename T, int N>
int scan_launch(ScanArgs a, cudaStream_t st) {
  using C = LongCfg<N>;
  const int sms = a.g.sms;
  const bool any_long = a.g.T > kShortTokens && a.g.T > a.g.S;
  if (any_long) {
    ScanArgs l = a;
    l.short_max = kShortTokens;
    l.blocks = a.channels / a.per_group * ((a.per_group + C::CPW - 1) / C::CPW);
    // one CTA an SM stays, and each has a task before one has two
    const int64_t tasks = (max_long(a.g.T, a.g.S) + a.slots) * l.blocks;
    const int64_t grid = tasks < sms ? tasks : sms;
    if (const int e = allow_smem<scan_long_kernel<T, N, true>>(C::kSmem)) return e;
    if (const int e = allow_smem<scan_long_kernel<T, N, false>>(C::kSmem)) return e;
    if (const int e = launch_beside(scan_long_kernel<T, N, true>, false, grid, 32 * C::kWarps, C::kSmem, st, l))
      return e;
    if (l.piece > 0) {
      const int64_t quads = static_cast<int64_t>(a.channels) * N / 4;
      if (const int e = launch_beside(scan_carry_kernel<N>, true, (quads + kCarryThreads - 1) / kCarryThreads,
                                      kCarryThreads, 0, st, l))
        return e;
      if (const int e = launch_beside(scan_long_kernel<T, N, false>, true, grid, 32 * C::kWarps, C::kSmem, st, l))
        return e;
    }
  }
  // without the long kernel this one takes segments of any length
  a.short_max = any_long ? kShortTokens : 0x7fffffff;
  constexpr int per = ShortCfg<N>::CPW;
  a.blocks = (a.channels + per - 1) / per;
  // more warps than stay at once (32 an SM), as a warp's last segments end
  // unevenly; for little work one round of them, whose starts are not repeated
  // (8192 channels, 28 and 64 warps an SM: 16 segments 7.3 and 7.9 us, 64 17.1 and
  // 16.9, 128 30.7 and 27.0, 256 54.0 and 48.6)
  const int64_t per_sm = static_cast<int64_t>(a.blocks) * a.g.S < 256LL * sms ? 28 : 64;
  const int64_t want = (per_sm * sms + a.blocks - 1) / a.blocks;
  a.split = static_cast<int32_t>(want < a.g.S ? want : a.g.S);
  const int64_t warps = static_cast<int64_t>(a.blocks) * a.split;
  const int64_t grid = (warps + kShortThreads / 32 - 1) / (kShortThreads / 32) + 1;
  return launch_beside(scan_short_kernel<T, N>, any_long, grid, kShortThreads, 0, st, a);
}
template <typename T>
int scan_states(const ScanArgs& a, int N, cudaStream_t st) {
  if (N == 8) return scan_launch<T, 8>(a, st);
  if (N == 16) return scan_launch<T, 16>(a, st);
  if (N == 32) return scan_launch<T, 32>(a, st);
  return scan_launch<T, 64>(a, st);
}

// How a convolution is dealt out: tokens of a run, runs, CTAs across the channels.
struct ConvCut {
  int32_t tokens, runs, blocks;
  int64_t grid;
};
ConvCut conv_cut(const mcp_conv_desc& d) {
  ConvCut c;
  c.blocks = (d.channels / kConvCh + kConvThreads - 1) / kConvThreads;
  // runs: long ones read fewer inputs twice (K - 1 in TT), shorter ones keep
  // every SM busy when the stream is short
  for (c.tokens = kConvMaxRun;; c.tokens /= 2) {
    c.runs = (d.total_tokens + c.tokens - 1) / c.tokens;
    if (c.tokens == 8 || static_cast<int64_t>(c.runs) * c.blocks >= 4 * step_num_sms()) break;
  }
  if (d.total_tokens <= kShortTokens) c.runs = 0;
  c.grid = ((d.num_seqs + kPack - 1) / kPack + static_cast<int64_t>(c.runs)) * c.blocks + 1;
  return c;
}

}  // namespace

bool mixed_conv_fits(const mcp_conv_desc& d) {
  const ConvCut c = conv_cut(d);  // a bound on the grid: a CTA a segment
  return (d.num_seqs + static_cast<int64_t>(c.runs)) * c.blocks < 0x7fffffff;
}

int launch_mixed_conv(const mcp_conv_desc& d, const void* x, const void* weight, const void* bias,
                      void* state, const int32_t* request_ids, const int32_t* cu_seqlens_q,
                      const int32_t* seqlens_k, void* out, int32_t* error_word, void* stream) {
  ConvArgs a;
  a.g = {request_ids, cu_seqlens_q, seqlens_k, d.num_seqs, d.total_tokens, d.num_requests, error_word,
         step_num_sms()};
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.state = state;
  a.out = out;
  a.ldx = d.x_stride;
  a.ldo = d.out_stride;
  a.channels = d.channels;
  a.act = d.activation;
  const ConvCut cut = conv_cut(d);
  a.tokens = cut.tokens;
  a.runs = cut.runs;
  a.blocks = cut.blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d.dtype == MCP_DTYPE_BF16 ? conv_width<__nv_bfloat16>(a, d.width, cut.grid, st)
                                   : conv_width<__half>(a, d.width, cut.grid, st);
}

size_t mixed_scan_workspace(const mcp_scan_desc& d, int sms) { return scan_cut(d, sms).bytes; }

bool mixed_scan_fits(const mcp_scan_desc& d) {
  const int sms = step_num_sms();
  const int64_t tasks = (max_long(d.total_tokens, d.num_seqs) + scan_cut(d, sms).slots) * long_blocks(d);
  return tasks + static_cast<int64_t>(sms) * long_warps(d.state_size) < 0x7fffffff;
}

int launch_mixed_scan(const mcp_scan_desc& d, const mcp_scan_tensors& t,
                      const int32_t* request_ids, const int32_t* cu_seqlens_q,
                      const int32_t* seqlens_k, void* workspace, int32_t* error_word,
                      void* stream) {
  ScanArgs a = {};
  a.g = {request_ids, cu_seqlens_q, seqlens_k, d.num_seqs, d.total_tokens, d.num_requests, error_word,
         step_num_sms()};
  a.x = t.x;
  a.dt = t.dt;
  a.A = t.A;
  a.B = t.B;
  a.C = t.C;
  a.D = t.D;
  a.z = t.z;
  a.dt_bias = t.dt_bias;
  a.state = t.state;
  a.out = t.out;
  a.ldx = d.x_stride;
  a.lddt = d.dt_stride;
  a.ldz = d.z_stride;
  a.ldb = d.b_stride;
  a.ldc = d.c_stride;
  a.ldo = d.out_stride;
  a.channels = d.channels;
  a.per_group = d.channels / d.num_groups;
  a.softplus = d.softplus;
  const ScanCut cut = scan_cut(d, step_num_sms());
  if (workspace && cut.piece > 0) {
    a.piece = cut.piece;
    a.slots = cut.slots;
    a.counter = static_cast<int32_t*>(workspace);
    a.carries = reinterpret_cast<float*>(static_cast<char*>(workspace) + 256);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d.dtype == MCP_DTYPE_BF16 ? scan_states<__nv_bfloat16>(a, d.state_size, st)
                                   : scan_states<__half>(a, d.state_size, st);
}

}  // namespace mcp
