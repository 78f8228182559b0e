// Verification of drafted tokens against the target's probabilities.
//
// A segment's rows are the nodes of a tree; node i was drafted under node
// parents[i].  From the root on, the nodes under the current one are tried in
// order.  With the probabilities q that they were drawn from, what is left of p
// after some were refused is r(v) = max(p(v) - c q(v), 0) / N: refusing another
// makes max(r - q, 0) = max(p - (c + N) q, 0) / N of it, so c grows by N and N is
// the new sum; the whole history of refusals is two numbers.  Without q a refused
// token's p becomes 0.  The walk ends where no node is left, and the last token is
// the first v whose prefix sum passes u times the sum.
//
// What this takes: the nodes' probabilities are two dependent loads, all nodes at
// once; the walk itself reads shared memory; then one pass over the row (over p
// and q) where the walk ends, another for every refusal after which a node is left
// to try, and a second look at the few hundred values in which the prefix sum
// passes.  A cluster of CTAs shares a segment: each sums a part of the row, and the
// parts' sums go to every CTA of the cluster through distributed shared memory.
//
// The token that comes out is a whole number, and each of the vocabulary's
// borders is a chance to round to another one: with sums off by a part of d that is
// about 2 V d a token, 1% with the 2^-24 of fp32 at V = 128000.  Values and sums are
// therefore pairs of fp32, about 2^-46 (fp64 would take the pass from its loads to
// the fp64 unit: 2 a clock and SM).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxNodes = 1024;

// ------------------------------------------------------- sums of two fp32
struct Two {
  float h, l;
};
// a + b exactly, as a sum and its error
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two normal(float h, float l) {  // |h| >= |l|
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.h, b.h);
  return normal(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ bool above(Two a, Two b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
__device__ __forceinline__ double wide(Two a) { return static_cast<double>(a.h) + a.l; }
__device__ __forceinline__ Two two_of(double x) {
  const float h = static_cast<float>(x);
  return {h, static_cast<float>(x - h)};
}

// ------------------------------------------------------------ probabilities
template <typename T>
__device__ __forceinline__ float as_float(T x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
  else return __bfloat162float(x);
}
// entries that are negative, infinite or NaN count as 0
__device__ __forceinline__ float clean(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};
template <typename T>
__device__ __forceinline__ void unpack(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      } else {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
}

struct VerifyArgs {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu;
  const float* u;
  const float* u_last;
  int32_t* accepted;
  int32_t* path;
  int32_t* out;
  int32_t* err;
  int64_t ldp, ldq;
  int32_t S, R, V;
};

// The weights of one row: p, p - c q, or p without some tokens.
template <typename T, bool kDraft>
struct Row {
  const T* p;
  const T* q;          // kDraft
  float ch, cl;        // c as two fp32
  const int32_t* gone;  // tokens whose weight is 0 (!kDraft)
  int num_gone;

  __device__ __forceinline__ Two weight(float p_raw, float q_raw) const {
    const float pv = clean(p_raw);
    if constexpr (!kDraft) {
      return {pv, 0.f};
    } else {
      const float qv = clean(q_raw);
      // p - (ch + cl) q: the product and the difference each with its error
      const float t = __fmul_rn(ch, qv), e = __fmaf_rn(ch, qv, -t);
      const Two d = two_sum(pv, -t);
      const Two w = normal(d.h, __fsub_rn(__fsub_rn(d.l, e), __fmul_rn(cl, qv)));
      return w.h > 0.f ? w : Two{0.f, 0.f};
    }
  }
  __device__ __forceinline__ bool is_gone(int v) const {
    for (int i = 0; i < num_gone; ++i)
      if (gone[i] == v) return true;
    return false;
  }
  // weight of token v, read alone
  __device__ __forceinline__ Two at(int v) const {
    if (!kDraft && num_gone && is_gone(v)) return {0.f, 0.f};
    return weight(as_float(p[v]), kDraft ? as_float(q[v]) : 0.f);
  }
};

__device__ __forceinline__ void accumulate(Two& acc, Two w) {
  const Two s = two_sum(acc.h, w.h);
  acc.h = s.h;
  acc.l = __fadd_rn(acc.l, __fadd_rn(s.l, w.l));
}

// Sum of the weights of tokens [a, b) over the lanes of a warp, each holding its
// part.  `off`: element of its 16 bytes at which row p (and q) begins, or < 0
// when p and q begin at different ones and are read value by value.
template <typename T, bool kDraft>
__device__ __forceinline__ Two lane_sum(const Row<T, kDraft>& r, int64_t a, int64_t b, int off, int lane) {
  constexpr int N = Vec<T>::N, kAhead = 4;
  Two acc = {0.f, 0.f};
  bool some_gone = false;
  if constexpr (!kDraft) {  // a few parts of the row hold refused tokens
    bool mine = false;
    for (int i = lane; i < r.num_gone; i += 32) mine |= r.gone[i] >= a && r.gone[i] < b;
    some_gone = __any_sync(0xffffffffu, mine);
  }
  if (off >= 0 && !some_gone) {
    // whole 16-byte pieces, counted from the one that holds the row's first value
    const int64_t first = (a + off + N - 1) / N, last = (b + off) / N;  // inside [a, b)
    const uint4* pv = reinterpret_cast<const uint4*>(r.p - off);
    const uint4* qv = kDraft ? reinterpret_cast<const uint4*>(r.q - off) : nullptr;
    for (int64_t k = first + lane; k < last; k += 32 * kAhead) {
      uint4 wp[kAhead], wq[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool in = k + 32 * j < last;
        wp[j] = in ? __ldg(pv + k + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
        if (kDraft) wq[j] = in ? __ldg(qv + k + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        float x[N], y[N];
        unpack<T>(wp[j], x);
        if (kDraft) unpack<T>(wq[j], y);
#pragma unroll
        for (int i = 0; i < N; ++i) accumulate(acc, r.weight(x[i], kDraft ? y[i] : 0.f));
      }
    }
    // the values before and behind the whole pieces
    const int64_t head = first * N - off < b ? first * N - off : b;
    const int64_t tail = last * N - off > head ? last * N - off : head;
    for (int64_t v = a + lane; v < head; v += 32) accumulate(acc, r.at(static_cast<int>(v)));
    for (int64_t v = tail + lane; v < b; v += 32) accumulate(acc, r.at(static_cast<int>(v)));
  } else {
    for (int64_t v = a + lane; v < b; v += 32 * kAhead) {
      float x[kAhead], y[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool in = v + 32 * j < b;
        x[j] = in ? as_float(r.p[v + 32 * j]) : 0.f;
        y[j] = kDraft && in ? as_float(r.q[v + 32 * j]) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (kDraft || !some_gone || !r.is_gone(static_cast<int>(v + 32 * j)))
          accumulate(acc, r.weight(x[j], y[j]));
    }
  }
  return normal(acc.h, acc.l);
}

__device__ __forceinline__ Two warp_sum(Two a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Two b = {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
    // the same order of operands on both sides: one result in all lanes
    a = (threadIdx.x & o) ? add(b, a) : add(a, b);
  }
  return a;
}
__device__ __forceinline__ Two warp_scan(Two a, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two b = {__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
    if (lane >= o) a = add(b, a);
  }
  return a;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// store two fp32 at the place of `local` in the shared memory of CTA `rank`
__device__ __forceinline__ void store_remote(const Two* local, uint32_t rank, Two x) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  asm volatile(
      "{\n.reg .b32 r;\nmapa.shared::cluster.u32 r, %0, %1;\n"
      "st.shared::cluster.v2.f32 [r], {%2, %3};\n}" ::"r"(a), "r"(rank), "f"(x.h), "f"(x.l)
      : "memory");
}

struct Shared {
  Two sums[2][kMaxCluster * kWarps];  // of the row's parts, two calls' worth
  float pt[kMaxNodes], qt[kMaxNodes], u[kMaxNodes];
  int32_t tok[kMaxNodes];
  int16_t par[kMaxNodes];
  int32_t gone[kMaxNodes];
  int32_t num_gone;
  // the walk's state
  int32_t cur, next, kept;
  int32_t need;    // another node waits for N
  int32_t refused;  // a node under cur was refused since N
  double c, N;
  // the place where the prefix sum passes
  Two scan[kWarps];
  int32_t last, hit;
};

// The walk from where it stands until it ends or needs a sum; one warp.  `out`
// and `path` are written where `lead` (one CTA of the cluster).
template <bool kDraft>
__device__ __forceinline__ void walk(Shared& sh, const VerifyArgs& p, int r0, int n, bool lead, int lane) {
  int cur = sh.cur, i = sh.next, kept = sh.kept;
  double c = sh.c, N = sh.N;
  bool refused = sh.refused;
  int need = 0;
  while (true) {
    int found = -1;
    for (int b = i; b < n && found < 0; b += 32) {
      const unsigned m = __ballot_sync(0xffffffffu, b + lane < n && sh.par[b + lane] == cur);
      if (m) found = b + __ffs(m) - 1;
    }
    if (found < 0) break;
    i = found;
    const double pv = sh.pt[i], u = sh.u[i];
    const int tok = sh.tok[i];
    bool ok, again = false;
    if constexpr (kDraft) {
      if (refused) {  // N of the new residual first
        need = 1;
        break;
      }
      const double qv = sh.qt[i];
      ok = __dmul_rn(__dmul_rn(u, N), qv) < __dsub_rn(pv, __dmul_rn(c, qv));
    } else {
      // a token that was already refused under this node has no weight left
      if (refused)
        for (int b = cur + 1; b < i; b += 32)
          again |= b + lane < i && sh.par[b + lane] == cur && sh.tok[b + lane] == tok;
      again = __any_sync(0xffffffffu, again);
      ok = !again && __dmul_rn(u, N) < pv;
    }
    if (ok) {
      if (lead && lane == 0) {
        p.path[r0 + kept] = i;
        p.out[r0 + kept - 1] = tok;
      }
      ++kept;
      cur = i;
      c = 0.0;
      N = 1.0;
      refused = false;
    } else {
      if (kDraft) c += N;
      else if (!again) N = N > pv ? N - pv : 0.0;
      refused = true;
    }
    ++i;
  }
  __syncwarp();
  if (lane == 0) {
    sh.cur = cur;
    sh.next = i;
    sh.kept = kept;
    sh.c = c;
    sh.N = N;
    sh.refused = refused;
    sh.need = need;
  }
}

template <typename T, bool kDraft>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int s = blockIdx.x / C;
  const bool lead = rank == 0;
  const int r0 = p.cu[s], r1 = p.cu[s + 1], n = r1 - r0;
  if (n <= 0 || r0 < 0 || r1 > p.R || n > kMaxNodes) {  // the same in all CTAs of the cluster
    if (lead && tid == 0) {
      p.accepted[s] = 0;
      if (n != 0 && p.err) atomicOr(p.err, MCP_DEVERR_SEGMENT);
    }
    return;
  }
  const T* const P = static_cast<const T*>(p.target);
  const T* const Q = static_cast<const T*>(p.draft);
  // every node's token under its parent's rows
  int bad = 0;
  for (int i = tid; i < n; i += kThreads) {
    const int t = p.tokens[r0 + i];
    int a = i == 0 ? -1 : p.parents ? p.parents[r0 + i] : i - 1;
    if (a >= i && i > 0) {
      bad |= MCP_DEVERR_TREE;
      a = -1;
    }
    if (i > 0 && t >= p.V) bad |= MCP_DEVERR_TOKEN_RANGE;
    if (t < 0 || t >= p.V) a = -1;
    float pv = 0.f, qv = 0.f;
    if (a >= 0) {
      pv = clean(as_float(P[(r0 + a) * p.ldp + t]));
      if (kDraft) qv = clean(as_float(Q[(r0 + a) * p.ldq + t]));
    }
    sh.par[i] = static_cast<int16_t>(a < 0 ? -1 : a);
    sh.tok[i] = t;
    sh.pt[i] = pv;
    sh.qt[i] = qv;
    sh.u[i] = p.u[r0 + i];
  }
  if (lead && bad && p.err) atomicOr(p.err, bad);
  if (tid == 0) {
    sh.cur = 0;
    sh.next = 1;
    sh.kept = 1;
    sh.c = 0.0;
    sh.N = 1.0;
    sh.refused = 0;
    sh.num_gone = 0;
    if (lead) p.path[r0] = 0;
  }
  // every CTA of the cluster runs before another writes to its shared memory
  if (C == 1) __syncthreads();
  else cluster_sync();

  // the part of a row that this warp sums: pieces of 32 bytes and more
  const int parts = C * kWarps;
  const int64_t per = ((static_cast<int64_t>(p.V) + parts - 1) / parts + 15) / 16 * 16;
  const int part = rank * kWarps + warp;
  const int64_t a = per * part < p.V ? per * part : p.V, b = a + per < p.V ? a + per : p.V;
  int calls = 0;
  Row<T, kDraft> row;
  int off = 0;
  // sum of the weights of row `cur`, in all CTAs; the parts' sums are in sh.sums[calls & 1]
  auto pass = [&](int cur, double c) -> Two {
    row.p = P + (r0 + cur) * p.ldp;
    row.q = kDraft ? Q + (r0 + cur) * p.ldq : nullptr;
    const Two cc = two_of(c);
    row.ch = cc.h;
    row.cl = cc.l;
    const int op = static_cast<int>((reinterpret_cast<uintptr_t>(row.p) & 15) / sizeof(T));
    const int oq = static_cast<int>((reinterpret_cast<uintptr_t>(row.q) & 15) / sizeof(T));
    off = !kDraft || op == oq ? op : -1;
    const Two mine = warp_sum(lane_sum<T, kDraft>(row, a, b, off, lane));
    Two* sums = sh.sums[++calls & 1];
    if (C == 1) {
      if (lane == 0) sums[part] = mine;
      __syncthreads();
    } else {
      if (lane < C) store_remote(sums + part, lane, mine);
      cluster_sync();
    }
    Two t = {0.f, 0.f};
    for (int k = lane; k < parts; k += 32) t = add(t, sums[k]);
    return warp_sum(t);
  };

  row.gone = sh.gone;
  row.num_gone = 0;
  while (true) {
    if (warp == 0) walk<kDraft>(sh, p, r0, n, lead, lane);
    __syncthreads();
    if (!kDraft || !sh.need) break;
    const Two t = pass(sh.cur, sh.c);
    __syncthreads();  // everybody has read the walk's state
    if (tid == 0) {
      sh.N = wide(t);
      sh.refused = 0;
    }
    __syncthreads();
  }
  const int cur = sh.cur, kept = sh.kept;
  if constexpr (!kDraft) {  // the refused tokens: all that hang under the last node
    for (int i = tid; i < n; i += kThreads)
      if (sh.par[i] == cur) sh.gone[atomicAdd(&sh.num_gone, 1)] = sh.tok[i];
    __syncthreads();
    row.num_gone = sh.num_gone;
  }
  Two total = pass(cur, sh.c);
  if (!(total.h > 0.f)) {  // nothing remains: the target's row itself
    row.num_gone = 0;
    total = pass(cur, 0.0);
  }
  if (lead) {  // places behind the path
    for (int i = kept + tid; i < n; i += kThreads) {
      p.path[r0 + i] = -1;
      p.out[r0 + i] = -1;
    }
    if (tid == 0) p.accepted[s] = kept;
  }
  int32_t* const answer = p.out + r0 + kept - 1;
  if (!(total.h > 0.f)) {
    if (lead && tid == 0) {
      *answer = -1;
      if (p.err) atomicOr(p.err, MCP_DEVERR_PROBS);
    }
    return;
  }
  // the part in which the prefix sum passes u * total (every warp for itself): the
  // first whose end is above it, else the last that holds anything
  const Two aim = two_of(static_cast<double>(p.u_last[s]) * wide(total));
  const Two* sums = sh.sums[calls & 1];
  int in = -1, last = 0;
  Two before = {0.f, 0.f}, at_last = {0.f, 0.f};
  for (int k0 = 0; k0 < parts && in < 0; k0 += 32) {
    const int k = k0 + lane;
    const Two x = k < parts ? sums[k] : Two{0.f, 0.f};
    const Two incl = add(before, warp_scan(x, lane));
    const unsigned m = __ballot_sync(0xffffffffu, x.h > 0.f && above(incl, aim));
    const unsigned some = __ballot_sync(0xffffffffu, x.h > 0.f);
    const int at = m ? __ffs(m) - 1 : some ? 31 - __clz(some) : -1;
    if (at >= 0) {  // the sum before part `at`
      const Two up = {__shfl_sync(0xffffffffu, incl.h, at ? at - 1 : 0),
                      __shfl_sync(0xffffffffu, incl.l, at ? at - 1 : 0)};
      at_last = at ? up : before;
      last = k0 + at;
    }
    if (m) in = last;
    before = {__shfl_sync(0xffffffffu, incl.h, 31), __shfl_sync(0xffffffffu, incl.l, 31)};
  }
  if (in < 0) in = last;
  if (in / kWarps != rank) return;
  // this CTA's threads take a piece of the part each, in order
  const int64_t a1 = per * in, b1 = a1 + per < p.V ? a1 + per : p.V;
  const int64_t each = (per + kThreads - 1) / kThreads;
  const int64_t v0 = a1 + each * tid < b1 ? a1 + each * tid : b1, v1 = v0 + each < b1 ? v0 + each : b1;
  if (tid == 0) {
    sh.last = -1;
    sh.hit = 0x7fffffff;
  }
  Two mine = {0.f, 0.f};
  int32_t positive = -1;
  for (int64_t v = v0; v < v1; ++v) {
    const Two w = row.at(static_cast<int>(v));
    if (w.h > 0.f) positive = static_cast<int32_t>(v);
    accumulate(mine, w);
  }
  mine = normal(mine.h, mine.l);
  const Two inside = warp_scan(mine, lane);
  const Two ahead = {__shfl_up_sync(0xffffffffu, inside.h, 1), __shfl_up_sync(0xffffffffu, inside.l, 1)};
  if (lane == 31) sh.scan[warp] = inside;
  __syncthreads();
  Two base = at_last;
  for (int w = 0; w < warp; ++w) base = add(base, sh.scan[w]);
  const bool passes = positive >= 0 && above(add(base, inside), aim);
  if (passes) atomicMin(&sh.hit, tid);
  if (positive >= 0) atomicMax(&sh.last, positive);
  __syncthreads();
  if (sh.hit == 0x7fffffff) {  // u = 1, or the sums' last bits
    if (tid == 0) *answer = sh.last;
    return;
  }
  if (sh.hit != tid) return;
  Two run = lane ? add(base, ahead) : base;
  int32_t found = positive;
  for (int64_t v = v0; v < v1; ++v) {
    const Two w = row.at(static_cast<int>(v));
    run = add(run, w);
    if (w.h > 0.f && above(run, aim)) {
      found = static_cast<int32_t>(v);
      break;
    }
  }
  *answer = found;
}

// CTAs that share a segment: as many as the GPU has room for at once (two a SM),
// but none with less than 4096 values of a row.
int cluster_of(const mcp_verify_desc& d) {
  int c = kMaxCluster;
  while (c > 1 && (static_cast<int64_t>(d.num_seqs) * c > 2LL * step_num_sms() || d.vocab_size / c < 4096))
    c /= 2;
  return c;
}

template <typename T>
int launch_typed(const mcp_verify_desc& d, const VerifyArgs& a, void* stream) {
  cudaLaunchAttribute at = {};
  const int c = cluster_of(d);
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(c);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(d.num_seqs * c));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return static_cast<int>(a.draft ? cudaLaunchKernelEx(&cfg, verify_kernel<T, true>, a)
                                  : cudaLaunchKernelEx(&cfg, verify_kernel<T, false>, a));
}

}  // namespace

int launch_verify_drafts(const mcp_verify_desc& d, const mcp_verify_tensors& t, int32_t* error_word,
                         void* stream) {
  VerifyArgs a;
  a.target = t.target;
  a.draft = t.draft;
  a.tokens = t.tokens;
  a.parents = t.parents;
  a.cu = t.cu_rows;
  a.u = t.uniform;
  a.u_last = t.final_uniform;
  a.accepted = t.accepted;
  a.path = t.path;
  a.out = t.new_tokens;
  a.err = error_word;
  a.ldp = d.target_stride;
  a.ldq = d.draft_stride;
  a.S = d.num_seqs;
  a.R = d.total_rows;
  a.V = d.vocab_size;
  if (d.dtype == MCP_DTYPE_BF16) return launch_typed<__nv_bfloat16>(d, a, stream);
  if (d.dtype == MCP_DTYPE_FP16) return launch_typed<__half>(d, a, stream);
  return launch_typed<float>(d, a, stream);
}

}  // namespace mcp
