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
// therefore pairs of fp32 (fp64 would take the pass from its loads to the fp64 unit: 2 a
// clock and SM): a weight is off by 2^-47 of p + c q at most, a sum of 128000 values by about
// 2^-45 of itself and one of 2^22 by 2^-41, since a lane's low words are added up in fp32.
// What remains after refusals is a part of p and c q and keeps the fewer bits the smaller it is.
//
// Measured: 64 chains of 4 to 8 rows of 128000 fp32 values (65 MB of p and q where the
// walks end) 18.8 us, the pass itself at 5.5 TB/s behind 5 us of loads that depend on
// each other; 32 trees of up to 32 rows, the mean of three sets of them, some with eight
// passes, 31.6; 256 given trees of 50257 bf16 values 20.5 (26 MB,
// bound by the latencies and the sums' operations); one chain 7.4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "mcp.h"
#include "step_ops.h"

namespace mcp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxNodes = 1024;
constexpr int kGoneBits = 65536;  // of the bitmap of refused tokens
constexpr int kSlots = 8;         // 16-byte pieces that a thread has in flight
constexpr int kSlotsGiven = 6;    // without q, where the bitmap takes the room of two
constexpr int kPerSM = 4;         // CTAs

// ------------------------------------------------------- sums of two fp32
struct Two {
  float h, l;
};
// a + b exactly, as a sum and its error
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two normal(Two a) {  // |h| >= |l|
  const float s = __fadd_rn(a.h, a.l);
  return {s, __fsub_rn(a.l, __fsub_rn(s, a.h))};
}
// the sum, whose l may have grown past half a step of h
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.h, b.h);
  return {s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}
__device__ __forceinline__ bool above(Two a, Two b) {  // of normal ones
  return a.h > b.h || (a.h == b.h && a.l > b.l);
}
__device__ __forceinline__ double wide(Two a) { return static_cast<double>(a.h) + a.l; }
__device__ __forceinline__ Two two_of(double x) {
  const float h = static_cast<float>(x);
  return {h, static_cast<float>(x - h)};
}
// acc += w for w >= 0 and acc.h >= 0: with the larger first, the error of the sum
// takes two operations instead of four
__device__ __forceinline__ void accumulate(Two& acc, float w) {
  const float a = fmaxf(acc.h, w), b = fminf(acc.h, w);
  const float s = __fadd_rn(a, b);
  acc.l = __fadd_rn(acc.l, __fsub_rn(b, __fsub_rn(s, a)));
  acc.h = s;
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

// What a weight is made of: p, p - q after one refusal, p - c q after several.
enum Mode : int { kOnlyP = 0, kLessQ = 1, kLessCQ = 2 };

// The weights of one row
template <typename T>
struct Row {
  const T* p;
  const T* q;
  int mode;
  float ch, cl;         // c as two fp32
  const int32_t* gone;  // tokens whose weight is 0
  int num_gone;
  const uint32_t* bitmap;  // bit (place % kGoneBits): the token there may be one of them
  int off;                 // place of token 0: values of its 16-byte piece before it
  bool folded;             // the places are more than the bits: the list decides

  __device__ __forceinline__ bool is_gone(int64_t place) const {
    const uint32_t f = static_cast<uint32_t>(place) % kGoneBits;
    if (!(bitmap[f >> 5] >> (f & 31) & 1u)) return false;
    if (!folded) return true;
    for (int i = 0; i < num_gone; ++i)
      if (gone[i] + off == place) return true;
    return false;
  }
};

// max(p - (ch + cl) q, 0) of probabilities p and q as a sum of two fp32.  c q is t + lo, |lo|
// up to 1.5 units of t's last place: where p is that close to t (p - t is exact there) lo
// says whether p - c q is positive, and may be all of it.
__device__ __forceinline__ Two less_cq(float pv, float qv, float ch, float cl) {
  const float t = __fmul_rn(ch, qv), lo = __fmaf_rn(cl, qv, __fmaf_rn(ch, qv, -t));
  const float d = __fsub_rn(pv, t);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(pv, d), t), lo);  // d + e = p - c q
  const float all = __fadd_rn(d, e);
  return {fmaxf(all, 0.f), all > 0.f ? __fsub_rn(e, __fsub_rn(all, d)) : 0.f};
}
// The same of values as they stand there, so that a part whose sum is positive holds a
// positive value.  Not inlined: the kernel waits for instructions more than for anything
// else where they are run once a row.
__device__ __noinline__ Two weight_of(float p_raw, float q_raw, float ch, float cl) {
  return less_cq(clean(p_raw), clean(q_raw), ch, cl);
}
// Weight of token v, read alone
template <typename T>
__device__ __forceinline__ Two weight_at(const Row<T>& r, int v) {
  if (r.num_gone && r.is_gone(static_cast<int64_t>(v) + r.off)) return {0.f, 0.f};
  if (r.mode == kOnlyP) return {clean(as_float(r.p[v])), 0.f};
  return weight_of(as_float(r.p[v]), as_float(r.q[v]), r.ch, r.cl);
}

// Weights of tokens v .. v + 3 (0 from `end` on), their loads in flight together
template <typename T>
__device__ __forceinline__ void weights_at(const Row<T>& r, int64_t v, int64_t end, Two* x) {
  float pv[4], qv[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = v + j < end;
    pv[j] = in ? as_float(r.p[v + j]) : 0.f;
    qv[j] = in && r.mode != kOnlyP ? as_float(r.q[v + j]) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = r.mode == kOnlyP ? Two{clean(pv[j]), 0.f} : weight_of(pv[j], qv[j], r.ch, r.cl);
    if (r.num_gone && r.is_gone(v + j + r.off)) x[j] = {0.f, 0.f};
  }
}

__device__ __forceinline__ void copy_async(uint4* to, const uint4* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from)
               : "memory");
}
// The largest bits of `worst` and a piece, and whether they are of a value that is
// negative, infinite or NaN (those have the largest): one operation for two values
template <typename T>
__device__ __forceinline__ uint32_t worst_of(uint32_t worst, uint4 w) {
  if constexpr (std::is_same_v<T, float>)
    return __vimax3_u32(__vimax3_u32(worst, w.x, w.y), w.z, w.w);
  else
    return __vimax3_u16x2(__vimax3_u16x2(worst, w.x, w.y), w.z, w.w);
}
template <typename T>
__device__ __forceinline__ bool no_probability(uint32_t worst) {
  if constexpr (std::is_same_v<T, float>) return worst >= 0x7f800000u;
  constexpr uint32_t kInf = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
  return (worst >> 16) >= kInf || (worst & 0xffffu) >= kInf;
}

// Sum of the weights of tokens [a, b) over the lanes of a warp, each holding its
// part.  `off`: element of its 16 bytes at which row p (and q) begins, or < 0 when
// p and q begin at different ones and are read value by value.
//
// p and q are taken as they stand, and their bits' maximum tells whether one of
// them was negative, infinite or NaN (1 operation a value where setting those to 0
// takes 2): then the part is summed again value by value.  max(p, q) - q instead of
// max(p - q, 0) leaves no error to be cleared.
template <typename T, int kMode, int kRing>
__device__ __forceinline__ Two lane_sum(const Row<T>& r, int64_t a, int64_t b, int off, int lane,
                                        uint4* ring) {
  constexpr int N = Vec<T>::N;
  Two acc = {0.f, 0.f};
  uint32_t worst = 0;  // of 16-bit types: of both halves
  auto take = [&](float pv, float qv) {
    if constexpr (kMode == kOnlyP) {
      accumulate(acc, pv);
    } else {
      float w, e;
      if constexpr (kMode == kLessQ) {
        const float m = fmaxf(pv, qv);
        w = __fsub_rn(m, qv);
        e = __fsub_rn(__fsub_rn(m, w), qv);
      } else {
        const Two x = less_cq(pv, qv, r.ch, r.cl);
        w = x.h;
        e = x.l;
      }
      accumulate(acc, w);
      acc.l = __fadd_rn(acc.l, e);
    }
  };
  int64_t head = b, tail = b;  // [a, head) and [tail, b) are read value by value
  if (off >= 0) {
    // whole 16-byte pieces, counted from the one that holds the row's first value.
    // A thread copies its own to shared memory, kDepth of them ahead of the one it
    // adds up: in registers, four pieces of p and q ahead left the SM waiting for
    // memory between rounds.
    constexpr int kDepth = kMode == kOnlyP ? kRing : kRing / 2;
    const int64_t first = (a + off + N - 1) / N, last = (b + off) / N;  // inside [a, b)
    head = min(first * N - off, b);
    tail = max(last * N - off, head);
    const int count = static_cast<int>(max(last - first, static_cast<int64_t>(0)));
    const uint4* pv = reinterpret_cast<const uint4*>(r.p - off) + first + lane;
    const uint4* qv = kMode == kOnlyP ? nullptr : reinterpret_cast<const uint4*>(r.q - off) + first + lane;
    uint4* const slot = ring + threadIdx.x;
    int ahead = lane;  // the piece to be fetched next
    auto fetch = [&](int at) {
      if (ahead < count) {
        copy_async(slot + at * kThreads, pv);
        if (kMode != kOnlyP) copy_async(slot + (kDepth + at) * kThreads, qv);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ahead += 32;
      pv += 32;
      if (kMode != kOnlyP) qv += 32;
    };
#pragma unroll
    for (int j = 0; j < kDepth - 1; ++j) fetch(j);
    for (int k = lane; k < count;) {
#pragma unroll
      for (int at = 0; at < kDepth; ++at) {  // the slots in turn
        if (k >= count) break;
        fetch((at + kDepth - 1) % kDepth);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        const uint4 wp = slot[at * kThreads];
        uint4 wq = make_uint4(0u, 0u, 0u, 0u);
        if (kMode != kOnlyP) wq = slot[(kDepth + at) * kThreads];
        worst = worst_of<T>(worst, wp);
        if (kMode != kOnlyP) worst = worst_of<T>(worst, wq);
        float x[N], y[N];
        unpack<T>(wp, x);
        if (kMode != kOnlyP) unpack<T>(wq, y);
        if (kMode == kOnlyP && r.num_gone) {
          const int64_t place = (first + k) * N;  // of the piece's first value, N bits of one word
          const uint32_t f = static_cast<uint32_t>(place) % kGoneBits;
          if (r.bitmap[f >> 5] >> (f & 31) & ((1u << N) - 1u)) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (r.is_gone(place + i)) x[i] = 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) take(x[i], kMode == kOnlyP ? 0.f : y[i]);
        k += 32;
      }
    }
  }
  bool odd = no_probability<T>(worst);
#pragma unroll 1
  for (int64_t v = a + lane; v < b; v += 32) {
    if (v >= head && v < tail) {  // on to the first of this lane's that is behind the pieces
      v += (tail - v + 31) / 32 * 32;
      if (v >= b) break;
    }
    if (kMode == kOnlyP && r.num_gone && r.is_gone(v + r.off)) continue;
    const float x = as_float(r.p[v]), y = kMode == kOnlyP ? 0.f : as_float(r.q[v]);
    odd |= __float_as_uint(x) >= 0x7f800000u || __float_as_uint(y) >= 0x7f800000u;
    take(x, y);
  }
  if (__any_sync(0xffffffffu, odd)) {  // by all lanes, which share the part anew
    acc = {0.f, 0.f};
#pragma unroll 1
    for (int64_t v = a + lane; v < b; v += 32) {
      const Two w = weight_at(r, static_cast<int>(v));
      accumulate(acc, w.h);
      acc.l = __fadd_rn(acc.l, w.l);
    }
  }
  return acc;
}

// Sum over groups of kLanes lanes, the same bits in all of them
template <int kLanes>
__device__ __forceinline__ Two lanes_sum(Two a) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)  // two_sum and + do not depend on the operands' order
    a = add(a, {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)});
  return a;
}
// Inclusive prefix sums over groups of kLanes lanes
template <int kLanes>
__device__ __forceinline__ Two lanes_scan(Two a, int lane) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const Two b = {__shfl_up_sync(0xffffffffu, a.h, o, kLanes), __shfl_up_sync(0xffffffffu, a.l, o, kLanes)};
    if ((lane & (kLanes - 1)) >= o) a = add(b, a);
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
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// store two fp32 at the place of `local` in the shared memory of CTA `rank`
__device__ __forceinline__ void store_remote(const Two* local, uint32_t rank, Two x) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  asm volatile(
      "{\n.reg .b32 r;\nmapa.shared::cluster.u32 r, %0, %1;\n"
      "st.shared::cluster.v2.f32 [r], {%2, %3};\n}" ::"r"(a), "r"(rank), "f"(x.h), "f"(x.l)
      : "memory");
}

template <bool kDraft>
struct Shared {
  static constexpr int kRing = kDraft ? kSlots : kSlotsGiven;
  uint4 ring[kRing * kThreads];
  uint32_t bitmap[kDraft ? 4 : kGoneBits / 32];
  Two sums[2][kMaxCluster];  // of the CTAs' parts of the row, two passes' worth
  Two part[kWarps];          // of this CTA's warps'
  float pt[kMaxNodes], u[kMaxNodes];
  union {
    float qt[kMaxNodes];      // with q
    int32_t gone[kMaxNodes];  // without
  };
  int32_t tok[kMaxNodes];
  int16_t par[kMaxNodes];
  bool first_ok[kMaxNodes];  // accepted if it is the first that is tried under its parent
  int32_t num_gone;
  // the pass that is asked for: row, c, and whether the walk is over
  int32_t cur, kept, over;
  Two c;
  // the part in which the prefix sum passes (-1: none of this CTA's), the sum before
  // it, and what its threads found
  int32_t in, last, hit;
  Two start, aim;
  Two scan[kWarps];
};

// Where a walk stands; the same in all lanes of the warp that walks
struct Walk {
  int cur = 0, next = 1, kept = 1;
  double c = 0.0, N = 1.0;
  bool refused = false;  // a node under cur was refused (with q: since N)
};

// On until the walk ends (true) or needs N of what is left (false).  `out` and
// `path` are written where `lead` (one CTA of the cluster).
template <bool kDraft>
__device__ __forceinline__ bool walk(Walk& w, const Shared<kDraft>& sh, const VerifyArgs& p, int r0, int n, bool lead,
                                     int lane) {
#pragma unroll 1
  for (int base = w.next & ~31; base < n; base += 32) {
    const int par = base + lane < n ? sh.par[base + lane] : -1;
    const unsigned first_ok = __ballot_sync(0xffffffffu, base + lane < n && sh.first_ok[base + lane]);
#pragma unroll 1
    while (true) {
      const int from = w.next - base;
      const unsigned m = __ballot_sync(0xffffffffu, par == w.cur) & (from < 32 ? ~0u << from : 0u);
      if (!m) break;
      const int i = base + __ffs(m) - 1;
      const int tok = sh.tok[i];
      bool ok, again = false;
      if (kDraft && w.refused) return false;  // N of the new residual first
      if (kDraft ? w.c == 0.0 : !w.refused) {
        ok = first_ok >> (i & 31) & 1u;
      } else if constexpr (kDraft) {
        const double qv = sh.qt[i];
        ok = __dmul_rn(__dmul_rn(sh.u[i], w.N), qv) < __dsub_rn(sh.pt[i], __dmul_rn(w.c, qv));
      } else {
        // a token that was already refused under this node has no weight left
        for (int b = w.cur + 1; b < i; b += 32)
          again |= b + lane < i && sh.par[b + lane] == w.cur && sh.tok[b + lane] == tok;
        again = __any_sync(0xffffffffu, again);
        ok = !again && __dmul_rn(sh.u[i], w.N) < sh.pt[i];
      }
      w.next = i + 1;
      w.refused = !ok;
      if (ok) {
        if (lead && lane == 0) {
          p.path[r0 + w.kept] = i;
          p.out[r0 + w.kept - 1] = tok;
        }
        ++w.kept;
        w.cur = i;
        w.c = 0.0;
        w.N = 1.0;
      } else if (kDraft) {
        w.c += w.N;
      } else if (!again) {
        const double pv = sh.pt[i];
        w.N = w.N > pv ? w.N - pv : 0.0;
      }
    }
    w.next = max(w.next, base + 32);
  }
  return true;
}

template <typename T, bool kDraft>
__global__ void __launch_bounds__(kThreads, kPerSM) verify_kernel(const VerifyArgs p) {
  extern __shared__ __align__(16) unsigned char smem[];
  using Sh = Shared<kDraft>;
  Sh& sh = *reinterpret_cast<Sh*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int s = blockIdx.x / C;
  const bool lead = rank == 0;
  const int r0 = p.cu[s], r1 = p.cu[s + 1];
  // compared as they are: the difference of wild bounds leaves 32 bits
  if (r1 <= r0 || r0 < 0 || r1 > p.R || r1 - r0 > kMaxNodes) {  // the same in all CTAs of the cluster
    if (lead && tid == 0) {
      p.accepted[s] = 0;
      if (r1 != r0 && p.err) atomicOr(p.err, MCP_DEVERR_SEGMENT);
    }
    return;
  }
  const int n = r1 - r0;
  const float u_last = p.u_last[s];
  if (C > 1) cluster_arrive_relaxed();  // this CTA runs; waited for before the first remote write
  const T* const P = static_cast<const T*>(p.target);
  const T* const Q = static_cast<const T*>(p.draft);
  // every node's token under its parent's rows
  int bad = 0;
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) {
    const int t = p.tokens[r0 + i];
    int a = i == 0 ? -1 : p.parents ? p.parents[r0 + i] : i - 1;
    const float u = p.u[r0 + i];
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
    if (kDraft) sh.qt[i] = qv;
    sh.u[i] = u;
    // u q < p: the product's error decides where it rounds to p
    const float uq = kDraft ? __fmul_rn(u, qv) : u;
    sh.first_ok[i] = uq < pv || (kDraft && uq == pv && __fmaf_rn(u, qv, -uq) < 0.f);
  }
  if (lead && bad && p.err) atomicOr(p.err, bad);
  if (tid == 0) {
    sh.num_gone = 0;
    if (lead) p.path[r0] = 0;
  }
  __syncthreads();

  // A row is cut into parts of whole 16-byte pieces, counted from the piece that holds
  // its first value (`off` values before that one): a warp's part ends inside a piece
  // only where the row does
  const int64_t per = ((static_cast<int64_t>(p.V) + 16 + C * kWarps - 1) / (C * kWarps) + 15) / 16 * 16;
  auto begin_of = [&](int64_t part, int off) {
    return min(max(per * part - max(off, 0), static_cast<int64_t>(0)), static_cast<int64_t>(p.V));
  };
  Row<T> row;
  row.gone = sh.gone;
  row.num_gone = 0;
  row.bitmap = sh.bitmap;
  row.folded = static_cast<int64_t>(p.V) + 16 > kGoneBits;
  Walk w;
  bool over = false;
  Two total;
  int passes = 0, off = 0;
  // Warp 0 walks and says which row is to be summed; all warps sum; until the walk is
  // over and something remains where it ended.
  while (true) {
    if (warp == 0) {
      if (!over) over = walk<kDraft>(w, sh, p, r0, n, lead, lane);
      if (lane == 0) {
        sh.cur = w.cur;
        sh.kept = w.kept;
        sh.c = two_of(w.c);
        sh.over = over;
      }
    }
    __syncthreads();
    const int cur = sh.cur;
    const Two c = sh.c;
    over = sh.over;
    row.p = P + (r0 + cur) * p.ldp;
    row.q = kDraft ? Q + (r0 + cur) * p.ldq : nullptr;
    row.mode = !kDraft || c.h == 0.f ? kOnlyP : c.h == 1.f && c.l == 0.f ? kLessQ : kLessCQ;
    row.ch = c.h;
    row.cl = c.l;
    const int op = static_cast<int>((reinterpret_cast<uintptr_t>(row.p) & 15) / sizeof(T));
    if constexpr (!kDraft) {
      if (passes == 0) {  // the refused tokens: all that hang under the last node
        for (int i = tid; i < kGoneBits / 128; i += kThreads)
          reinterpret_cast<uint4*>(sh.bitmap)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (int i = tid; i < n; i += kThreads)
          if (sh.par[i] == cur) {
            sh.gone[atomicAdd(&sh.num_gone, 1)] = sh.tok[i];
            const uint32_t f = static_cast<uint32_t>(sh.tok[i] + op) % kGoneBits;
            atomicOr(&sh.bitmap[f >> 5], 1u << (f & 31));
          }
        __syncthreads();
        row.num_gone = sh.num_gone;
      } else {
        row.num_gone = 0;  // nothing remained: the target's row itself
      }
    }
    off = op;
    if (kDraft && row.mode != kOnlyP && op != static_cast<int>((reinterpret_cast<uintptr_t>(row.q) & 15) / sizeof(T)))
      off = -1;
    row.off = op;
    const int64_t a = begin_of(rank * kWarps + warp, off), b = begin_of(rank * kWarps + warp + 1, off);
    Two mine;
    if constexpr (kDraft) {
      mine = row.mode == kOnlyP ? lane_sum<T, kOnlyP, Sh::kRing>(row, a, b, off, lane, sh.ring)
             : row.mode == kLessQ ? lane_sum<T, kLessQ, Sh::kRing>(row, a, b, off, lane, sh.ring)
                                  : lane_sum<T, kLessCQ, Sh::kRing>(row, a, b, off, lane, sh.ring);
    } else {
      mine = lane_sum<T, kOnlyP, Sh::kRing>(row, a, b, off, lane, sh.ring);
    }
    mine = lanes_sum<32>(mine);
    if (lane == 0) sh.part[warp] = normal(mine);
    __syncthreads();
    // the CTA's sum to every CTA of the cluster, all of which run by now (the first
    // wait); two passes' sums are kept, so that no CTA writes what another still reads
    Two* sums = sh.sums[passes & 1];
    if (C > 1 && passes == 0) cluster_wait();
    if (warp == 0) {
      const Two all = normal(lanes_sum<kWarps>(sh.part[lane & (kWarps - 1)]));
      if (C == 1) {
        if (lane == 0) sums[0] = all;
      } else if (lane < C) {
        store_remote(sums + rank, lane, all);
      }
    }
    if (C == 1) {
      __syncthreads();
    } else {
      if (warp == 0) cluster_arrive();
      else cluster_arrive_relaxed();
      cluster_wait();
    }
    ++passes;
    const int k = lane & (kMaxCluster - 1);
    total = normal(lanes_sum<kMaxCluster>(k < C ? sums[k] : Two{0.f, 0.f}));
    if (!over) {
      w.N = wide(total);
      w.refused = false;
    } else {
      if (total.h > 0.f || (row.mode == kOnlyP && row.num_gone == 0)) break;
      w.c = 0.0;  // nothing remains: the target's row itself
    }
  }
  const int kept = sh.kept;
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
  if (warp == 0) {
    // the part in which the prefix sum passes u * total: the first whose end is above
    // it, else the last that holds anything
    const float aim_h = __fmul_rn(u_last, total.h);
    const Two aim = normal({aim_h, __fmaf_rn(u_last, total.l, __fmaf_rn(u_last, total.h, -aim_h))});
    Two start = {0.f, 0.f};
    int in = -1;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {  // among the CTAs, then among this one's warps
      const Two* of = level ? sh.part : sh.sums[(passes - 1) & 1];
      const Two x = lane < (level ? kWarps : C) ? of[lane] : Two{0.f, 0.f};
      const Two incl = normal(add(start, lanes_scan<16>(x, lane)));
      const unsigned m = __ballot_sync(0xffffffffu, x.h > 0.f && above(incl, aim));
      const unsigned some = __ballot_sync(0xffffffffu, x.h > 0.f);
      in = m ? __ffs(m) - 1 : some ? 31 - __clz(some) : 0;
      const Two up = {__shfl_sync(0xffffffffu, incl.h, in ? in - 1 : 0),
                      __shfl_sync(0xffffffffu, incl.l, in ? in - 1 : 0)};
      if (in) start = up;
      if (level == 0 && in != rank) {
        in = -1;
        break;
      }
    }
    if (lane == 0) {
      sh.in = in;
      sh.start = start;
      sh.aim = aim;
      sh.last = -1;
      sh.hit = 0x7fffffff;
    }
  }
  __syncthreads();
  if (sh.in < 0) return;
  // this CTA's threads take a piece of the part each, in order
  const Two aim = sh.aim;
  const int64_t a1 = begin_of(rank * kWarps + sh.in, off), b1 = begin_of(rank * kWarps + sh.in + 1, off);
  const int64_t each = (per + kThreads - 1) / kThreads;
  const int64_t v0 = min(a1 + each * tid, b1), v1 = min(v0 + each, b1);
  Two mine = {0.f, 0.f};
  int32_t positive = -1;
#pragma unroll 1
  for (int64_t v = v0; v < v1; v += 4) {
    Two x[4];
    weights_at(row, v, v1, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (x[j].h > 0.f) positive = static_cast<int32_t>(v) + j;
      accumulate(mine, x[j].h);
      mine.l = __fadd_rn(mine.l, x[j].l);
    }
  }
  const Two inside = lanes_scan<32>(mine, lane);
  const Two ahead = {__shfl_up_sync(0xffffffffu, inside.h, 1), __shfl_up_sync(0xffffffffu, inside.l, 1)};
  if (lane == 31) sh.scan[warp] = inside;
  __syncthreads();
  const Two warps = lanes_scan<kWarps>(sh.scan[lane & (kWarps - 1)], lane);
  const Two up = {__shfl_sync(0xffffffffu, warps.h, warp ? warp - 1 : 0),
                  __shfl_sync(0xffffffffu, warps.l, warp ? warp - 1 : 0)};
  const Two base = warp ? add(sh.start, up) : sh.start;
  if (positive >= 0) {
    if (above(normal(add(base, inside)), aim)) atomicMin(&sh.hit, tid);
    atomicMax(&sh.last, positive);
  }
  __syncthreads();
  if (sh.hit == 0x7fffffff) {  // u = 1, or the sums' last bits
    if (tid == 0) *answer = sh.last;
    return;
  }
  if (sh.hit != tid) return;
  Two run = lane ? add(base, ahead) : base;
  int32_t found = -1;
#pragma unroll 1
  for (int64_t v = v0; v < v1 && found < 0; v += 4) {
    Two x[4];
    weights_at(row, v, v1, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      run = add(run, x[j]);
      if (found < 0 && x[j].h > 0.f && above(normal(run), aim)) found = static_cast<int32_t>(v) + j;
    }
  }
  *answer = found >= 0 ? found : positive;
}

// CTAs that share a segment: as many as the GPU has room for at once, but none with
// less than 4096 values of a row.  With 4, 8 and 16 of them 64 chains take 22.9, 18.9 and
// 25.8 us, one chain 14.2, 9.5 and 7.5, 32 trees 50, 36.6 and 31.6; with 1, 2 and 4 256 given
// trees 22.8, 20.6 and 24.6.
int cluster_of(const mcp_verify_desc& d) {
  int c = kMaxCluster;
  while (c > 1 && (static_cast<int64_t>(d.num_seqs) * c > kPerSM * static_cast<int64_t>(step_num_sms()) || d.vocab_size / c < 4096))
    c /= 2;
  return c;
}

// Clusters of more than 8 CTAs have to be asked for, once per kernel and device.
template <auto kernel>
int allow_large_clusters() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return 0;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return static_cast<int>(e);
}

template <typename T, bool kDraft>
int launch_typed(const mcp_verify_desc& d, const VerifyArgs& a, void* stream) {
  int e = allow_smem<verify_kernel<T, kDraft>>(sizeof(Shared<kDraft>));
  if (e != 0) return e;
  const int c = cluster_of(d);
  if (c > 8) {
    e = allow_large_clusters<verify_kernel<T, kDraft>>();
    if (e != 0) return e;
  }
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(c);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(d.num_seqs * c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared<kDraft>);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, verify_kernel<T, kDraft>, a));
}

template <typename T>
int launch_either(const mcp_verify_desc& d, const VerifyArgs& a, void* stream) {
  return a.draft ? launch_typed<T, true>(d, a, stream) : launch_typed<T, false>(d, a, stream);
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
  if (d.dtype == MCP_DTYPE_BF16) return launch_either<__nv_bfloat16>(d, a, stream);
  if (d.dtype == MCP_DTYPE_FP16) return launch_either<__half>(d, a, stream);
  return launch_either<float>(d, a, stream);
}

}  // namespace mcp
