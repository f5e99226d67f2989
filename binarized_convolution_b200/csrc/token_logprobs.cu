// What rows of logits say (bconv_token_logprobs_*): log-sum-exp, entropy, the log probability of
// a given token and the top alternatives in one pass over the logits, and the gradient of log
// probability and entropy in another.
//
// With x = logits / temperature and m the largest logit seen, each thread keeps
//     s = sum exp((l - m) / temperature)     t = sum exp((l - m) / temperature) (l - m) / temperature
// over its elements (in powers of 2; rescaled when m grows), and these join pairwise, so a row is read once:
//     lse = m / temperature + log s          entropy = log s - t / s
// An element costs one fused multiply-add for the exponent, one exp2, one addition and one more
// multiply-add (see Stat).
//
// Top alternatives: the k-th largest of the maxima of disjoint groups of elements is a lower
// bound of the k-th largest element.  After its first batch of loads (32 elements a thread; fp32: 16), a CTA
// takes that bound from its threads' maxima, and from then on a thread only notes the batches whose largest
// element reaches it (few, unless the row is sorted).  At the end the threads' maxima of the whole part
// give a closer bound; what reaches it is collected from the noted batches and ordered by counting for each
// element how many come before it.  (Collecting elements while reading cost more than the reading: almost
// every batch of a warp holds one that reaches the first bound.)  Where the notes or the collected
// elements run over (sorted rows, long runs of equal logits), the part is read again with the closer bound,
// and if that does not suffice either, k passes over it pick one each.  Every path gives the
// same answer: logits in descending order, equal ones by index.
//
// A row is one CTA's work, or a cluster's where there are few rows; the cluster's CTAs hand their (m, s,
// t) and their own top k to the first one through its shared memory.
//
// Bound by HBM (one read of the logits; in the gradient one read and one write).
#include <float.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "dtype.cuh"
#include "f32x2.cuh"
#include "host_util.cuh"
#include "tc_device.cuh"

namespace bconv {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;          // CTAs an SM: enough that one's joins hide behind another's loads
constexpr int kMaxTop = 64;
constexpr int kCap = 1024;       // noted batches of one CTA, and elements collected from them
constexpr int kGroups = 128;     // groups of 2 threads whose maxima bound the k-th largest
constexpr int kMaxCluster = 8;
constexpr float kFar = -1e4f;    // exp2 of it and of anything below is 0; keeps 0 * d finite
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x by the hardware's approximation (relative error below 2^-22; -inf gives 0)
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order-preserving integer of a logit: larger values give larger keys, +-0 the same one, NaN the
// largest.  Keys are above 0, so 0 stands for "nothing".
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// (key, index) as one number that grows with the key and, for equal keys, falls with the index
__device__ __forceinline__ unsigned long long entry(uint32_t key, uint32_t index) {
  return (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ uint32_t entry_index(unsigned long long e) { return 0xffffffffu - static_cast<uint32_t>(e); }

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// s and t relative to the largest logit m, in powers of 2 of units c = log2(e) / temperature: an element v counts
// 2^d with d = v c - m c.  Usually ("near") m c is rounded once and v c - round(m c) is one exact
// multiply-add; that shifts all d by the same rounding, of at most 2^-5 for |m c| < 2^20, which drops out
// of every result as long as all use the same rounded product.  Beyond that the difference is taken first.
struct Stat {
  float m, s, t;
};

__device__ __forceinline__ bool near(float m, float c) { return fabsf(m * c) < 1048576.f && m > -1e30f; }

// d of an element v
__device__ __forceinline__ float relative(float v, float m, float c) {
  return near(m, c) ? fmaf(v, c, -__fmul_rn(m, c)) : (v - m) * c;
}

// The same relative to a larger m.
__device__ __forceinline__ void raise(Stat& a, float m, float c) {
  if (m > a.m) {
    float d = -FLT_MAX;  // with nothing but -inf so far s and t are 0 (or NaN, which stays)
    if (a.m != -INFINITY) {
      if (near(a.m, c)) d = near(m, c) ? __fsub_rn(__fmul_rn(a.m, c), __fmul_rn(m, c)) : fmaf(-m, c, __fmul_rn(a.m, c));
      else d = relative(a.m, m, c);
    }
    const float f = exp2_approx(d);
    a.t = fmaf(a.s, fmaxf(d, kFar), a.t) * f;
    a.s *= f;
    a.m = m;
  }
}
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
  raise(a, b.m, c);
  raise(b, a.m, c);
  return {a.m, a.s + b.s, a.t + b.t};
}
__device__ __forceinline__ Stat join_lanes(Stat st, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, st.t, o);
    st = join(st, b, c);
  }
  return st;
}

// A thread's running statistics: those of Stat with separate sums for even and odd elements.
struct Running {
  float m = -INFINITY, c, mc = 0.f;  // mc: m c rounded
  bool is_near = false;
  uint64_t s = 0, t = 0;
  __device__ __forceinline__ explicit Running(float c_) : c(c_) {}
  __device__ __forceinline__ Stat stat() const {
    const float2 a = unpair(s), b = unpair(t);
    return {m, a.x + a.y, b.x + b.y};
  }
  // Elements whose largest is mx (NaN if one is): first see, then add them.
  __device__ __forceinline__ void see(float mx) {
    if (mx > m) {
      Stat a = stat();
      raise(a, mx, c);
      m = mx;
      mc = __fmul_rn(m, c);
      is_near = near(m, c);
      s = pair(a.s, 0.f);
      t = pair(a.t, 0.f);
    }
  }
  template <int N>
  __device__ __forceinline__ void add_near(const float (&v)[N]) {
    const uint64_t cc = pair(c, c), mm = pair(-mc, -mc);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 d = unpair(fma2(pair(v[e], v[e + 1]), cc, mm));
      // (-inf: p = exp2(kFar) = 0, with a finite product)
      const float x = max_nan(d.x, kFar), y = max_nan(d.y, kFar);
      const uint64_t p = pair(exp2_approx(x), exp2_approx(y));
      s = add2(s, p);
      t = fma2(p, pair(x, y), t);
    }
  }
  __device__ __forceinline__ void add(float v) {
    if (v != -INFINITY) {
      const float d = max_nan(is_near ? fmaf(v, c, -mc) : (v - m) * c, kFar), p = exp2_approx(d);
      s = add2(s, pair(p, 0.f));
      t = fma2(pair(p, 0.f), pair(d, 0.f), t);
    }
  }
};

// A batch of a thread's steps (8 elements each) as they lie in memory: 64 bytes.
template <typename T>
struct Batch {
  static constexpr int kSteps = sizeof(T) == 2 ? 4 : 2;
  Raw8<T> w[kSteps];
  // Steps at, at + kThreads, ... of `steps`; -inf behind the last.
  __device__ __forceinline__ void load(const T* body, int at, int steps) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (at + i * kThreads < steps) {
        w[i].load(body + static_cast<int64_t>(at + i * kThreads) * 8);
      } else {
        float none[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) none[e] = -INFINITY;
        w[i].pack(none);
      }
    }
  }
  // The largest element, NaN if there is one: two at a time for the 16-bit types.
  __device__ __forceinline__ float largest() const {
    if constexpr (sizeof(T) == 2) {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 m = *reinterpret_cast<const T2*>(&w[0].w.x);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t u[4] = {w[i].w.x, w[i].w.y, w[i].w.z, w[i].w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = __hmax2_nan(m, *reinterpret_cast<const T2*>(&u[e]));
      }
      const float2 f = unpack2<T>(*reinterpret_cast<const uint32_t*>(&m));
      return max_nan(f.x, f.y);
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        float v[8];
        w[i].unpack(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, v[e]);
      }
      return m;
    }
  }
};

struct FwdArgs {
  const void* logits;
  const int64_t* tokens;
  float *logprob, *entropy, *lse, *top_logprob;
  int32_t* top_index;
  int64_t rows, stride;
  int vocab, top;
  float scale;  // 1 / temperature
  float c;      // log2(e) / temperature
};

struct Shared {
  Stat stat[kThreads / 32];
  Stat peers[kMaxCluster];                                  // first CTA: every CTA's statistics
  unsigned long long top[kMaxCluster * kMaxTop];            // first CTA: every CTA's top entries
  unsigned long long best[kThreads / 32];                   // one round of the slow selection
  unsigned long long noted[kCap];                           // batches that reach the bound: (key of the largest, first step)
  unsigned long long found[kCap];
  __align__(16) uint32_t group[kGroups];
  uint32_t bound;
  int batches, count;  // noted and found (counted on beyond the space)
};

// Element range [begin, end) of a row for a thread's loop: f(index, value) once for each element,
// 8 at a time from 16-byte aligned addresses, the ragged ends one at a time.
template <typename T, typename F8, typename F1>
__device__ __forceinline__ void each(const T* row, int begin, int end, F8&& f8, F1&& f1) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + begin);
  int head = static_cast<int>(((16 - (at & 15u)) & 15u) / sizeof(T));
  head = min(head, end - begin);
  const int body = (end - begin - head) / 8;
  const int tail = begin + head + body * 8;
  if (static_cast<int>(threadIdx.x) < head) f1(begin + threadIdx.x, to_f32(row[begin + threadIdx.x]));
  for (int i = threadIdx.x; i < body; i += kThreads) {
    Raw8<T> w;
    const int c = begin + head + i * 8;
    w.load(row + c);
    float v[8];
    w.unpack(v);
    f8(c, v);
  }
  if (tail + static_cast<int>(threadIdx.x) < end) f1(tail + threadIdx.x, to_f32(row[tail + threadIdx.x]));
}

// The `top`-th largest of the maxima of the CTA's groups of 2 threads, as a key (0 while
// fewer groups have seen an element).  `mx`: this thread's largest key, 0 for none.
__device__ __forceinline__ uint32_t bound_of(Shared& S, uint32_t mx, int top) {
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  if ((threadIdx.x & 1) == 0) S.group[threadIdx.x >> 1] = mx;
  if (threadIdx.x == 0) S.bound = 0;
  __syncthreads();
  if (threadIdx.x < kGroups) {
    const uint32_t own = S.group[threadIdx.x];
    int before = 0;
    const int at = threadIdx.x;
#pragma unroll 8
    for (int i = 0; i < kGroups; i += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&S.group[i]);
      before += (o.x > own || (o.x == own && i < at)) + (o.y > own || (o.y == own && i + 1 < at)) +
                (o.z > own || (o.z == own && i + 2 < at)) + (o.w > own || (o.w == own && i + 3 < at));
    }
    if (before == top - 1) S.bound = own;  // exactly one thread
  }
  __syncthreads();
  return S.bound;
}

__device__ __forceinline__ void collect(Shared& S, uint32_t key, int index) {
  const int at = atomicAdd(&S.count, 1);
  if (at < kCap) S.found[at] = entry(key, static_cast<uint32_t>(index));
}

// The largest `top` of n entries (distinct), in order, to out[0 .. top): counts for each how many come before.
__device__ __forceinline__ void order_entries(const unsigned long long* from, int n, int top, unsigned long long* out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long own = from[i];
    int before = 0;
    for (int j = 0; j < n; ++j) before += from[j] > own;
    if (before < top) out[before] = own;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) token_logprobs_fwd_kernel(const FwdArgs a) {
  __shared__ Shared S;
  uint32_t rank, peers;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(peers));
  const int64_t r = blockIdx.x / peers;
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  // this CTA's part of the row: whole 8-element steps
  const int part = static_cast<int>(((static_cast<int64_t>(a.vocab) + peers - 1) / peers + 7) / 8 * 8);
  const int begin = static_cast<int>(min(static_cast<int64_t>(rank) * part, static_cast<int64_t>(a.vocab)));
  const int end = static_cast<int>(min(static_cast<int64_t>(begin) + part, static_cast<int64_t>(a.vocab)));
  const int top = min(a.top, end - begin);  // this part's share of the candidates
  const float scale = a.scale, c2 = a.c;
  if (threadIdx.x == 0) S.count = S.batches = 0;
  // (awaited before the first access to another CTA's shared memory: that CTA has started by then)
  if (peers > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // the part as [head][body: 16-byte aligned, 8 elements a step][tail]; every thread has one element of head
  // and tail at most
  Running run(c2);
  const bool want = top > 0;
  const int head = min(end - begin, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(row + begin) & 15u)) & 15u) / sizeof(T)));
  const int steps = (end - begin - head) / 8, ends = end - begin - steps * 8;
  const T* const body = row + begin + head;
  const bool has_end = static_cast<int>(threadIdx.x) < ends;
  const int end_at = begin + static_cast<int>(threadIdx.x) + (static_cast<int>(threadIdx.x) < head ? 0 : steps * 8);
  float edge[1] = {-INFINITY};

  using B = Batch<T>;
  B now;
  now.load(body, threadIdx.x, steps);
  if (has_end) edge[0] = to_f32(row[end_at]);
  uint32_t bound = 0, most = has_end ? order_key(edge[0]) : 0u;  // most: this thread's largest
  float bound_value = -INFINITY;                                 // (NaN: every batch is noted)
  if (want) {  // the bound on the top entries, from the threads' first batches
    if (static_cast<int>(threadIdx.x) < steps) most = max(most, order_key(now.largest()));
    bound = bound_of(S, most, top);
    if (bound) bound_value = key_value(bound);
  }
  if (has_end) {
    run.see(edge[0]);
    run.add(edge[0]);
  }
  constexpr int kStride = B::kSteps * kThreads;
#pragma unroll 1
  for (int at = threadIdx.x; at < steps; at += kStride) {
    B next;
    next.load(body, at + kStride, steps);
    const float mx = now.largest();
    run.see(mx);
    if (run.is_near) {
#pragma unroll
      for (int i = 0; i < B::kSteps; ++i) {
        float v[8];
        now.w[i].unpack(v);
        run.add_near(v);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < B::kSteps; ++i) {
        float v[8];
        if (at + i * kThreads < steps) {
          Raw8<T> w;
          w.load(body + static_cast<int64_t>(at + i * kThreads) * 8);
          w.unpack(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) run.add(v[e]);
        }
      }
    }
    if (want && !(mx < bound_value)) {
      const uint32_t key = order_key(mx);
      most = max(most, key);
      const int note = atomicAdd(&S.batches, 1);
      if (note < kCap) S.noted[note] = (static_cast<unsigned long long>(key) << 32) | static_cast<uint32_t>(at);
    }
    now = next;
  }
  Stat st = run.stat();

  // statistics of the CTA
  st = join_lanes(st, c2);
  if ((threadIdx.x & 31) == 0) S.stat[threadIdx.x >> 5] = st;
  __syncthreads();

  // this part's top entries, in order, into the first CTA's shared memory
  if (want) {
    unsigned long long* mine = S.top;
    bound = bound_of(S, most, top);
    const int notes = S.batches;
    auto consider = [&](float v, int index) {
      const uint32_t k = order_key(v);
      if (k >= bound) collect(S, k, index);
    };
    if (has_end && notes <= kCap) consider(edge[0], end_at);
    if (notes <= kCap) {
      constexpr int kEach = B::kSteps * 8;
      for (int i = threadIdx.x; i < notes * kEach; i += kThreads) {
        const unsigned long long note = S.noted[i / kEach];
        if (static_cast<uint32_t>(note >> 32) < bound) continue;
        const int step = static_cast<int>(static_cast<uint32_t>(note)) + i % kEach / 8 * kThreads;
        if (step < steps) consider(to_f32(body[static_cast<int64_t>(step) * 8 + i % 8]), begin + head + step * 8 + i % 8);
      }
    } else {  // uniform
      each(row, begin, end,
           [&](int c, const float (&v)[8]) {
#pragma unroll
             for (int e = 0; e < 8; ++e) consider(v[e], c + e);
           },
           [&](int c, float v) { consider(v, c); });
    }
    __syncthreads();
    const int n = S.count;
    if (n <= kCap) {
      order_entries(S.found, n, top, mine);
    } else {  // one pass per entry: the largest below the last one
      unsigned long long last = ~0ull;
      for (int i = 0; i < top; ++i) {
        unsigned long long best = 0;
        each(row, begin, end,
             [&](int c, const float (&v)[8]) {
#pragma unroll
               for (int e = 0; e < 8; ++e) {
                 const unsigned long long x = entry(order_key(v[e]), static_cast<uint32_t>(c + e));
                 if (x < last && x > best) best = x;
               }
             },
             [&](int c, float v) {
               const unsigned long long x = entry(order_key(v), static_cast<uint32_t>(c));
               if (x < last && x > best) best = x;
             });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if ((threadIdx.x & 31) == 0) S.best[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) best = max(best, S.best[w]);
        __syncthreads();
        if (threadIdx.x == 0) mine[i] = best;
        last = best;
      }
    }
  }
  if (threadIdx.x < 32) {
    st = static_cast<int>(threadIdx.x) < kThreads / 32 ? S.stat[threadIdx.x] : Stat{-INFINITY, 0.f, 0.f};
    st = join_lanes(st, c2);
  }
  __syncthreads();
  int n = top;
  if (peers > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // every CTA's result to the first one (whose own entries are in place: peer p's start at p * a.top)
    if (rank != 0) {
      const uint32_t to = tcdev::mapa(&S.top[rank * a.top], 0), stat = tcdev::mapa(&S.peers[rank], 0);
      for (int i = threadIdx.x; i < a.top; i += kThreads) {
        const unsigned long long v = i < top ? S.top[i] : 0ull;
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + 8u * i), "l"(v) : "memory");
      }
      if (threadIdx.x == 0) {
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(stat), "f"(st.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(stat + 4u), "f"(st.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(stat + 8u), "f"(st.t) : "memory");
      }
    }
    __syncwarp();
    tcdev::cluster_sync();
    if (rank != 0) return;
    if (threadIdx.x == 0)
      for (uint32_t p = 1; p < peers; ++p) st = join(st, S.peers[p], c2);
    if (a.top > 0) {
      // entries of 0 ("nothing") come last: there are at least a.top real ones
      for (int i = threadIdx.x; i < static_cast<int>(peers) * a.top; i += kThreads) S.found[i] = i < a.top && i >= top ? 0ull : S.top[i];
      __syncthreads();
      order_entries(S.found, static_cast<int>(peers) * a.top, a.top, S.top);
    }
    n = a.top;
    __syncthreads();
  }
  if (threadIdx.x == 0) S.stat[0] = st;
  __syncthreads();
  st = S.stat[0];
  const bool nothing = st.m == -INFINITY && st.s == 0.f;
  const float log2_s = log2f(st.s);  // (the hardware's is off by 2^-22 near 1: nearly certain tokens)
  auto logprob = [&](float v) {
    if (st.s != st.s) return st.s;
    if (nothing || v == -INFINITY) return -INFINITY;
    const float d = relative(v, st.m, c2);
    return d < -1e30f ? (v - st.m) * scale : (d - log2_s) * kLn2;  // (far below: the product may have overflowed)
  };
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[r] = nothing ? -INFINITY : near(st.m, c2) ? (__fmul_rn(st.m, c2) + log2_s) * kLn2 : fmaf(st.m, scale, log2_s * kLn2);
    if (a.entropy) a.entropy[r] = nothing ? 0.f : (log2_s - st.t / st.s) * kLn2;
    if (a.logprob) {
      const int64_t token = a.tokens[r];
      a.logprob[r] = token < 0 ? 0.f : token >= a.vocab ? __uint_as_float(0x7fc00000u) : logprob(to_f32(row[token]));
    }
  }
  if (a.top_index && static_cast<int>(threadIdx.x) < n) {
    const unsigned long long x = S.top[threadIdx.x];
    a.top_index[r * a.top + threadIdx.x] = static_cast<int32_t>(entry_index(x));
    a.top_logprob[r * a.top + threadIdx.x] = logprob(key_value(static_cast<uint32_t>(x >> 32)));
  }
}

struct BwdArgs {
  const void* logits;
  const int64_t* tokens;
  const float *lse, *entropy, *d_logprob, *d_entropy;
  void* d_logits;
  int64_t rows, stride, d_stride;
  int vocab, parts;  // CTAs per row
  float scale;
};

constexpr int kBwdThreads = 256, kBwdBatch = 4;
constexpr int kBwdStep = kBwdThreads * 8 * kBwdBatch;  // elements of one CTA

template <typename T>
__global__ void __launch_bounds__(kBwdThreads) token_logprobs_bwd_kernel(const BwdArgs a) {
  const int64_t r = blockIdx.x / a.parts;
  const int begin = static_cast<int>(blockIdx.x - r * a.parts) * kBwdStep;
  const int end = min(a.vocab, begin + kBwdStep);
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  T* to = static_cast<T*>(a.d_logits) + r * a.d_stride;
  const bool vec = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(to)) & 15u) == 0;
  const int head = vec ? min(end - begin, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(row + begin) & 15u)) & 15u) / sizeof(T)))
                       : 0;
  const int steps = vec ? (end - begin - head) / 8 : 0, first = begin + head;
  Raw8<T> w[kBwdBatch];
#pragma unroll
  for (int i = 0; i < kBwdBatch; ++i) {
    const int at = static_cast<int>(threadIdx.x) + i * kBwdThreads;
    if (at < steps) w[i].load(row + first + at * 8);
  }
  const float scale = a.scale;
  const int64_t token = a.d_logprob ? a.tokens[r] : -1;
  float g = 0.f, ge = 0.f, h = 0.f, lse = a.lse[r];
  if (token >= 0) g = token < a.vocab ? a.d_logprob[r] : __uint_as_float(0x7fc00000u);
  if (a.d_entropy) {
    ge = a.d_entropy[r];
    h = a.entropy[r];
  }
  if (lse == -INFINITY) {  // nothing but -inf in the row: no gradient, at the token either (a NaN of g stays)
    lse = 0.f;
    g *= 0.f;
    ge *= 0.f;
  }
  // d = p (k0 + k1 log p), and g / temperature more at the token
  const float k0 = -(g + ge * h) * scale, k1 = -ge * scale;
  auto grad = [&](float v) {
    // (-inf: p = exp(kFar) = 0, with a finite product)
    const float logp = max_nan(fmaf(v, scale, -lse), kFar);
    return exp2_approx(logp * kLog2e) * fmaf(k1, logp, k0);
  };
  const float extra = g * scale;
#pragma unroll
  for (int i = 0; i < kBwdBatch; ++i) {
    const int at = static_cast<int>(threadIdx.x) + i * kBwdThreads;
    if (at < steps) {
      const int c = first + at * 8;
      float v[8];
      w[i].unpack(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = grad(v[e]);
      if (token >= c && token < c + 8)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e == token) v[e] += extra;
      w[i].pack(v);
      w[i].store(to + c);
    }
  }
  // the ragged ends (all of it where the rows' alignments differ)
  for (int i = threadIdx.x; i < end - begin - steps * 8; i += kBwdThreads) {
    const int c = i < head ? begin + i : begin + steps * 8 + i;
    float d = grad(to_f32(row[c]));
    if (c == token) d += extra;
    to[c] = from_f32<T>(d);
  }
}

// Whether operands of 4- and 8-byte elements (NULL allowed) are aligned to them.
bool aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return false;
  return true;
}
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

bconv_status_t check_desc(const bconv_token_desc_t* d) {
  if (!d || d->rows < 0 || d->rows > (int64_t{1} << 28) || d->vocab < 1 || d->vocab > (1 << 30) || d->stride < d->vocab ||
      !valid_dtype(d->dtype) || !(d->temperature > 0.f) || d->temperature > FLT_MAX || kLog2e / d->temperature > FLT_MAX)
    return BCONV_ERR_INVALID_ARG;
  return BCONV_OK;
}

template <typename T>
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s) {
  // CTAs per row: those that finish first, a CTA's fixed cost (the bound, the joins) being that of some
  // 8000 elements
  const int64_t slots = kCtas * static_cast<int64_t>(current_sm_count());
  unsigned peers = 1;
  double best = 1e300;
  for (unsigned p = 1; p <= kMaxCluster; p *= 2) {
    const double cost = static_cast<double>(ceil_div(a.rows * p, slots)) * (static_cast<double>(a.vocab) / p + 8000.0);
    if (cost < best * 0.98) {
      best = cost;
      peers = p;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * peers);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = peers;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, token_logprobs_fwd_kernel<T>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace bconv

using namespace bconv;

extern "C" {

bconv_status_t bconv_token_logprobs_forward(const bconv_token_desc_t* d, const void* logits, const int64_t* tokens,
                                            float* logprob, float* entropy, float* lse, float* top_logprob,
                                            int32_t* top_index, struct CUstream_st* stream) {
  const bconv_status_t st = check_desc(d);
  if (st != BCONV_OK) return st;
  if (d->top < 0 || d->top > kMaxTop || d->top > d->vocab || (logprob && !tokens) || !aligned_elem(logits, d->dtype) ||
      !aligned8(tokens) || !aligned4({logprob, entropy, lse, top_logprob, top_index}))
    return BCONV_ERR_INVALID_ARG;
  if (d->rows == 0) return BCONV_OK;
  if (!logits || (d->top > 0) != (top_logprob != nullptr) || (d->top > 0) != (top_index != nullptr))
    return BCONV_ERR_INVALID_ARG;
  FwdArgs a{logits, tokens, logprob, entropy, lse, top_logprob, top_index, d->rows, d->stride, d->vocab, d->top,
            1.f / d->temperature, kLog2e / d->temperature};
  return from_cuda(with_dtype(d->dtype, [&](auto t) { return launch_fwd<decltype(t)>(a, stream); }));
}

bconv_status_t bconv_token_logprobs_backward(const bconv_token_desc_t* d, const void* logits,
                                             const int64_t* tokens, const float* lse, const float* entropy,
                                             const float* d_logprob, const float* d_entropy, void* d_logits,
                                             int64_t d_stride, struct CUstream_st* stream) {
  const bconv_status_t st = check_desc(d);
  if (st != BCONV_OK) return st;
  if (d_stride < d->vocab || (d_logprob && !tokens) || (d_entropy && !entropy) || !aligned_elem(logits, d->dtype) ||
      !aligned_elem(d_logits, d->dtype) || !aligned8(tokens) || !aligned4({lse, entropy, d_logprob, d_entropy}) || (logits && logits == d_logits && d_stride != d->stride))
    return BCONV_ERR_INVALID_ARG;
  if (d->rows == 0) return BCONV_OK;
  if (!logits || !lse || !d_logits) return BCONV_ERR_INVALID_ARG;
  BwdArgs a{logits, tokens, lse, entropy, d_logprob, d_entropy, d_logits, d->rows, d->stride, d_stride, d->vocab,
            static_cast<int>(ceil_div(d->vocab, kBwdStep)), 1.f / d->temperature};
  const int64_t ctas = a.rows * a.parts;
  if (ctas > 0x7fffffff) return BCONV_ERR_UNSUPPORTED;
  return from_cuda(with_dtype(d->dtype, [&](auto t) {
    token_logprobs_bwd_kernel<decltype(t)><<<static_cast<unsigned>(ctas), kBwdThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }));
}

}  // extern "C"
