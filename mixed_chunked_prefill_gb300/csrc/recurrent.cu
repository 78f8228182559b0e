// The recurrent layers of a step over the packed stream: the short causal
// convolution and the selective state space scan, each segment continued from
// the state of its request and leaving its state for the next step.
//
// The stream is the one the mixed attention runs on ([W] "Flash Attention 的
// varlen 接口": decodes and chunks are segments of different lengths; the
// segment has history when seqlens_k counts more than its own tokens), so a
// decode is a segment of one token and a continued chunk starts from its
// request's state.  A segment's state is read and written by the one CTA (or
// thread) that owns its channels: no state crosses CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// ------------------------------------------------------------------ segments
struct Segments {
  const int32_t* ids;
  const int32_t* cu;
  const int32_t* sk;
  int32_t S, T, R;
  int32_t* err;
};

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
  const int32_t n = x.q1 - x.q0;
  x.old = g.sk[s] > n;
  if (x.q0 < 0 || n < 0 || x.q1 > g.T || x.id >= g.R) x.id = -1;
  return x;
}

// One CTA of each launch looks the metadata over: segments outside the stream,
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
// Each input is read once and each output written once; a thread carries the
// K - 1 last inputs of 8 channels (one 16-byte vector a token) in registers
// along a run of TT tokens, so only the first tokens of a run read inputs
// again.  HBM-bound for chunks; for decodes the K - 1 kept inputs of each
// request are read and written too and are most of the traffic.  The thread
// that runs over a segment's first token also runs over its next K - 2 (even
// past its run: those still need the kept inputs) and writes the new kept
// inputs, so nobody else reads or writes that state.
struct ConvArgs {
  Segments g;
  const void* x;
  const void* w;     // [channels, K]
  const void* bias;  // [channels] or NULL
  void* state;       // [R, K - 1, channels]
  void* out;
  int64_t ldx, ldo;
  int32_t channels, act, tokens, blocks;  // tokens: TT; blocks: CTAs across the channels
};

constexpr int kConvThreads = 128;
constexpr int kConvMaxRun = 16;

template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads) mixed_conv_kernel(const ConvArgs p) {
  if (blockIdx.x == 0) {
    check_segments(p.g);
    return;
  }
  constexpr int kBatch = 8;  // inputs requested together
  __shared__ Segment info[kConvMaxRun + K];
  __shared__ int32_t first;
  const int32_t tile = (blockIdx.x - 1) / p.blocks;
  const int32_t c = ((blockIdx.x - 1) % p.blocks * kConvThreads + threadIdx.x) * 8;
  const int32_t t0 = tile * p.tokens;
  const int32_t run = min(p.tokens, p.g.T - t0);
  const int32_t most = min(p.tokens + K - 2, p.g.T - t0);  // with a head that goes on
  // segments before the first token: those that end at or before it
  if (threadIdx.x == 0) first = 0;
  __syncthreads();
  int32_t n = 0;
  for (int32_t s = threadIdx.x; s < p.g.S; s += kConvThreads) n += p.g.cu[s + 1] <= t0;
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(&first, n);
  __syncthreads();
  if (threadIdx.x < most) {
    const int32_t t = t0 + threadIdx.x;
    int32_t lo = first, hi = p.g.S;  // first segment that ends behind t
    if (lo < hi && p.g.cu[lo + 1] <= t) {
      ++lo;
      while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (p.g.cu[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
      }
    }
    Segment x = {0, 0, -1, 0};
    if (lo < p.g.S) {
      x = read_segment(p.g, lo);
      if (t < x.q0 || t >= x.q1) x.id = -1;
    }
    info[threadIdx.x] = x;
  }
  __syncthreads();
  if (c >= p.channels) return;

  const uint4* X = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + c);
  uint4* O = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + c);
  const int64_t ldx = p.ldx / 8, ldo = p.ldo / 8, lds = p.channels / 8;
  float w[8 * K], b[8];  // w[i * K + k]: channel i, tap k (memory order)
#pragma unroll
  for (int k = 0; k < K; ++k)
    unpack8<T>(reinterpret_cast<const uint4*>(static_cast<const T*>(p.w) +
                                              static_cast<int64_t>(c) * K)[k], w + 8 * k);
  if (p.bias) {
    unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + c), b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.f;
  }
  float win[K - 1][8];
  bool have = false;  // win holds the K - 1 inputs before the next token
  for (int32_t i0 = 0; i0 < most; i0 += kBatch) {
    uint4 raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < most) raw[i] = X[(t0 + i0 + i) * ldx];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int32_t at = i0 + i;
      if (at >= most) break;
      const Segment s = info[at];
      const int32_t t = t0 + at, off = t - s.q0;
      // a segment's first K - 1 tokens belong to the run its first token is in
      const bool mine = s.id >= 0 && (off < K - 1 ? s.q0 >= t0 && s.q0 < t0 + run : at < run);
      if (!mine) {
        have = false;
        continue;
      }
      if (off == 0) {
        uint4* kept = reinterpret_cast<uint4*>(static_cast<T*>(p.state) +
                                               static_cast<int64_t>(s.id) * (K - 1) * p.channels + c);
        uint4 old[K - 1];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
          old[k] = s.old ? kept[k * lds] : make_uint4(0u, 0u, 0u, 0u);
          unpack8<T>(old[k], win[k]);
        }
        // the kept inputs of the next step: the last K - 1 of (old, segment)
        const int32_t len = s.q1 - s.q0;
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
          const int32_t from = len - (K - 1) + k;  // in the segment; < 0: old[K - 1 + from]
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (from >= 0) {
            v = X[(s.q0 + from) * ldx];
          } else {
#pragma unroll
            for (int m = 1; m < K - 1; ++m)
              if (K - 1 + from == m) v = old[m];
          }
          kept[k * lds] = v;
        }
      } else if (!have) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) unpack8<T>(X[(t - (K - 1) + k) * ldx], win[k]);
      }
      have = true;
      float v[8], y[8];
      unpack8<T>(raw[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a = b[e];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) a = fmaf(w[e * K + k], win[k][e], a);
        a = fmaf(w[e * K + K - 1], v[e], a);
        y[e] = p.act ? silu(a) : a;
      }
      O[t * ldo] = pack8<T>(y);
#pragma unroll
      for (int k = 0; k < K - 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) win[k][e] = win[k + 1][e];
#pragma unroll
      for (int e = 0; e < 8; ++e) win[K - 2][e] = v[e];
    }
  }
}

template <typename T, int K>
int conv_launch(const ConvArgs& a, int grid, cudaStream_t st) {
  mixed_conv_kernel<T, K><<<grid, kConvThreads, 0, st>>>(a);
  return static_cast<int>(cudaGetLastError());
}
template <typename T>
int conv_width(const ConvArgs& a, int K, int grid, cudaStream_t st) {
  if (K == 2) return conv_launch<T, 2>(a, grid, st);
  if (K == 3) return conv_launch<T, 3>(a, grid, st);
  return conv_launch<T, 4>(a, grid, st);
}

// --------------------------------------------------------------------- scan
// Per channel c and state n, along a segment's tokens:
//   d = softplus(dt + dt_bias),  h = exp(d A[c, n]) h + d x B[n],
//   y = sum_n C[n] h[c, n] + D[c] x,  out = y silu(z).
// State and sums are fp32.  exp(d A) is ex2.approx of d (A log2 e): 2 ulp,
// and the recurrence multiplies by it once a token.
//
// Least traffic: x, dt, z read and out written once (8 bytes per token and
// channel in 16 bits) and the states once.  One ex2 per token, channel and
// state: at the measured 32 a clock and SM, 16 states bound the kernel at
// 0.5 clocks per (token, channel), a little above the HBM time; the products
// run as packed pairs (two fp32 lanes an instruction) to stay below that.
//
// A lane holds 4 states of one channel in registers; N / 4 neighbouring lanes
// share a channel, 32 channels a CTA.  Tiles of 32 tokens go through shared
// memory: the thread that loads 8 channels of a token turns dt and x into
// (d, d x) there and keeps x and z in registers for its output, while the
// next tile's loads are in flight.  y's sums over the lanes of a channel are
// taken N / 4 tokens at a time (each exchange halves the tokens a lane
// carries), one shuffle a token instead of log2(N / 4).
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
  int32_t channels, per_group, softplus, blocks, split;  // split: CTAs the segments are dealt to
};

constexpr int kScanChannels = 32;
constexpr int kScanTile = 32;
constexpr float kLog2e = 1.44269504088896340736f;

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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// log(1 + exp(v)), to fp32's precision for small results too (log1p): the
// steps it gives may be 0.001 and less
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

template <typename T, int N>
__global__ void __launch_bounds__(8 * N) mixed_scan_kernel(const ScanArgs p) {
  if (blockIdx.x == 0) {
    check_segments(p.g);
    return;
  }
  constexpr int LPC = N / 4;                  // lanes of a channel
  constexpr int kThreads = kScanChannels * LPC;
  constexpr int kItems = kScanTile * 4;       // (token, 8 channels) of a tile
  constexpr int kPer = (kItems + kThreads - 1) / kThreads;
  constexpr int kYs = kScanChannels + (LPC <= 4 ? 32 / LPC : 4);  // a warp's stores spread over the banks
  __shared__ __align__(16) float2 dd[kScanTile][kScanChannels];
  __shared__ __align__(16) float bc[2][kScanTile][N];
  __shared__ __align__(16) float ys[kScanTile][kYs];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t cb = (blockIdx.x - 1) % p.blocks * kScanChannels;
  const int sub = lane % LPC, cl = (warp * 32 + lane) / LPC;  // states 4 sub.., channel of the block
  const int32_t c = cb + cl;
  const bool live = c < p.channels;
  const int32_t group = cb / p.per_group;

  f32x2 a01 = 0, a23 = 0;
  if (live) {
    const float4 a = *reinterpret_cast<const float4*>(p.A + static_cast<int64_t>(c) * N + 4 * sub);
    a01 = pack2(a.x * kLog2e, a.y * kLog2e);
    a23 = pack2(a.z * kLog2e, a.w * kLog2e);
  }
  // this thread's part of a tile: up to kPer (token, 8 channels) items and one
  // vector of B or C
  const int it_row = tid / 4, it_ch = (tid & 3) * 8;  // item i: row it_row + i * kThreads / 4
  const bool it_live = tid < kItems && cb + it_ch < p.channels;
  const int bc_which = tid / (4 * N), bc_row = tid % (4 * N) / (N / 8), bc_n = tid % (N / 8) * 8;
  const T* bc_src = static_cast<const T*>(bc_which ? p.C : p.B) + group * N + bc_n;
  const int64_t bc_ld = bc_which ? p.ldc : p.ldb;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

  for (int32_t s = (blockIdx.x - 1) / p.blocks; s < p.g.S; s += p.split) {
    const Segment seg = read_segment(p.g, s);
    const int32_t len = seg.q1 - seg.q0;
    if (seg.id < 0 || len == 0) continue;
    float* st = p.state + (static_cast<int64_t>(seg.id) * p.channels + c) * N + 4 * sub;
    f32x2 h01 = 0, h23 = 0;
    if (live && seg.old) {
      const float4 v = *reinterpret_cast<const float4*>(st);
      h01 = pack2(v.x, v.y);
      h23 = pack2(v.z, v.w);
    }
    uint4 rx[kPer], rd[kPer], rz[kPer], rb;
    auto load = [&](int32_t t0) {
      const int32_t left = seg.q1 - t0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = it_row + i * (kThreads / 4);
        const bool on = it_live && row < left;
        const int64_t t = t0 + row;
        const int64_t ch = cb + it_ch;
        rx[i] = on ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + t * p.ldx + ch) : zero;
        rd[i] = on ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.dt) + t * p.lddt + ch) : zero;
        rz[i] = on && p.z ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.z) + t * p.ldz + ch)
                          : zero;
      }
      rb = bc_row < left ? *reinterpret_cast<const uint4*>(bc_src + (t0 + bc_row) * bc_ld) : zero;
    };
    load(seg.q0);
    for (int32_t t0 = seg.q0; t0 < seg.q1; t0 += kScanTile) {
      const int32_t nt = min(kScanTile, seg.q1 - t0);
      uint4 cx[kPer], cz[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = it_row + i * (kThreads / 4);
        cx[i] = rx[i];
        cz[i] = rz[i];
        if (tid < kItems && row < ((nt + LPC - 1) & ~(LPC - 1))) {
          float x[8], d[8];
          unpack8<T>(rx[i], x);
          unpack8<T>(rd[i], d);
          float4* to = reinterpret_cast<float4*>(&dd[row][it_ch]);
          const bool on = it_live && row < nt;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (p.dt_bias && on) d[e] += p.dt_bias[cb + it_ch + e];
            if (p.softplus) d[e] = softplus(d[e]);
            if (!on) d[e] = 0.f;  // h stays: exp(0) h + 0
            x[e] *= d[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = make_float4(d[2 * e], x[2 * e], d[2 * e + 1], x[2 * e + 1]);
        }
      }
      {
        float f[8];
        unpack8<T>(rb, f);
        float4* to = reinterpret_cast<float4*>(&bc[bc_which][bc_row][bc_n]);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
      __syncthreads();
      if (t0 + kScanTile < seg.q1) load(t0 + kScanTile);
      for (int r0 = 0; r0 < nt; r0 += LPC) {
        float y[LPC];
#pragma unroll
        for (int i = 0; i < LPC; ++i) {
          const float2 d = dd[r0 + i][cl];
          const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&bc[0][r0 + i][4 * sub]);
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&bc[1][r0 + i][4 * sub]);
          const f32x2 dx = pack2(d.x, d.x), dy = pack2(d.y, d.y);
          float e0, e1, e2, e3;
          unpack2(mul2(dx, a01), e0, e1);
          unpack2(mul2(dx, a23), e2, e3);
          h01 = fma2(pack2(ex2(e0), ex2(e1)), h01, mul2(dy, b.x));
          h23 = fma2(pack2(ex2(e2), ex2(e3)), h23, mul2(dy, b.y));
          float y0, y1;
          unpack2(fma2(h01, q.x, mul2(h23, q.y)), y0, y1);
          y[i] = y0 + y1;
        }
        // lane bit k halves the tokens: the lane is left with the sum of one
        int row = r0;
#pragma unroll
        for (int w = LPC / 2, bit = 1; w >= 1; w >>= 1, bit <<= 1) {
          const bool up = lane & bit;
#pragma unroll
          for (int i = 0; i < w; ++i) {
            const float give = up ? y[i] : y[i + w], keep = up ? y[i + w] : y[i];
            y[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
          }
          if (up) row += w;
        }
        ys[row][cl] = y[0];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = it_row + i * (kThreads / 4);
        if (!it_live || row >= nt) continue;
        float x[8], z[8], y[8];
        unpack8<T>(cx[i], x);
        unpack8<T>(cz[i], z);
        const float4 lo = *reinterpret_cast<const float4*>(&ys[row][it_ch]);
        const float4 hi = *reinterpret_cast<const float4*>(&ys[row][it_ch + 4]);
        y[0] = lo.x, y[1] = lo.y, y[2] = lo.z, y[3] = lo.w;
        y[4] = hi.x, y[5] = hi.y, y[6] = hi.z, y[7] = hi.w;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (p.D) y[e] = fmaf(p.D[cb + it_ch + e], x[e], y[e]);
          if (p.z) y[e] *= silu(z[e]);
        }
        *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (t0 + row) * p.ldo + cb + it_ch) = pack8<T>(y);
      }
    }
    if (live) {
      float4 v;
      unpack2(h01, v.x, v.y);
      unpack2(h23, v.z, v.w);
      *reinterpret_cast<float4*>(st) = v;
    }
  }
}

template <typename T>
int scan_launch(const ScanArgs& a, int N, int grid, cudaStream_t st) {
  if (N == 8) mixed_scan_kernel<T, 8><<<grid, 64, 0, st>>>(a);
  else if (N == 16) mixed_scan_kernel<T, 16><<<grid, 128, 0, st>>>(a);
  else if (N == 32) mixed_scan_kernel<T, 32><<<grid, 256, 0, st>>>(a);
  else mixed_scan_kernel<T, 64><<<grid, 512, 0, st>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_mixed_conv(const mcp_conv_desc& d, const void* x, const void* weight, const void* bias,
                      void* state, const int32_t* request_ids, const int32_t* cu_seqlens_q,
                      const int32_t* seqlens_k, void* out, int32_t* error_word, void* stream) {
  ConvArgs a;
  a.g = {request_ids, cu_seqlens_q, seqlens_k, d.num_seqs, d.total_tokens, d.num_requests, error_word};
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.state = state;
  a.out = out;
  a.ldx = d.x_stride;
  a.ldo = d.out_stride;
  a.channels = d.channels;
  a.act = d.activation;
  a.blocks = (d.channels / 8 + kConvThreads - 1) / kConvThreads;
  // long runs read fewer inputs twice (K - 1 in TT), short ones keep every SM
  // busy when the stream is short
  int64_t tiles = 0;
  for (a.tokens = kConvMaxRun;; a.tokens /= 4) {
    tiles = (static_cast<int64_t>(d.total_tokens) + a.tokens - 1) / a.tokens;
    if (a.tokens == 1 || tiles * a.blocks >= 4 * step_num_sms()) break;
  }
  const int grid = static_cast<int>(tiles * a.blocks) + 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d.dtype == MCP_DTYPE_BF16 ? conv_width<__nv_bfloat16>(a, d.width, grid, st)
                                   : conv_width<__half>(a, d.width, grid, st);
}

int launch_mixed_scan(const mcp_scan_desc& d, const mcp_scan_tensors& t,
                      const int32_t* request_ids, const int32_t* cu_seqlens_q,
                      const int32_t* seqlens_k, int32_t* error_word, void* stream) {
  ScanArgs a;
  a.g = {request_ids, cu_seqlens_q, seqlens_k, d.num_seqs, d.total_tokens, d.num_requests, error_word};
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
  a.blocks = (d.channels + kScanChannels - 1) / kScanChannels;
  // enough CTAs for several per SM; more would only repeat the set-up
  const int64_t want = (32LL * step_num_sms() + a.blocks - 1) / a.blocks;
  a.split = static_cast<int32_t>(want < d.num_seqs ? want : d.num_seqs);
  const int grid = a.blocks * a.split + 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d.dtype == MCP_DTYPE_BF16 ? scan_launch<__nv_bfloat16>(a, d.state_size, grid, st)
                                   : scan_launch<__half>(a, d.state_size, grid, st);
}

}  // namespace mcp
