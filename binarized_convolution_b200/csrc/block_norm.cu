// What stands between two blocks of a language model (bconv_block_norm_*): the norm behind a
// block, its gate and residual scale, the residual sum and the norm before the next block, in
// one kernel per direction.
//
// Forward, per row of C channels (a = residual_scale, eps inside the root):
//     bs = rsqrt(mean(b^2) + eps);  p = b bs w_post;  r' = r + a g p
//     rs = rsqrt(mean(r'^2) + eps); n = r' rs w_pre
// Backward, from d_r' and d_n:
//     u = d_n w_pre;      dR = d_r' + rs (u - r' rs^2 mean(u r'))          -> d_r = dR
//     q = a g dR;         db = bs (q w_post - b bs^2 mean(q w_post b))     (no norm: db = q)
//     d_w_pre = sum_rows d_n r' rs;  d_w_post = sum_rows q b bs;  d_g = sum_rows a dR p
//
// The forward reads two and writes two arrays of rows x C, the backward reads four and writes two, all of
// them once.  One CTA holds a whole row (its threads 8 channels at a time), so each of the row sums is one block
// reduction.  Few, narrow or very wide rows take the plain kernels, which hold a row in registers; many rows of
// 257 to 8192 channels (the fp32 backward: to 5500, four arrays being all that two stages have room for) come ahead of
// their use through a ring in shared memory (below).
// With many rows HBM is kept 50 to 80 % busy: two reductions a row, each behind a barrier, and as many warps as
// the registers for sums and rows allow (4096 x 4096 bf16 backward: 128 registers, 15 warps an SM, which issue in 53 % of
// the cycles).  Rows in a graph, us: forward 8192 x 4096 bf16 53, 4096 x 4096 fp32 47 (5.7 TB/s); backward 4096 x 4096
// bf16 58, fp32 88 (4.6 TB/s), 8000 x 2001 bf16 61, 30000 x 384 bf16 51.
#include <algorithm>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "dtype.cuh"
#include "elect.cuh"
#include "f32x2.cuh"
#include "host_util.cuh"
#include "tc_device.cuh"

namespace bconv {
namespace {

constexpr int kMaxWidth = 32768;
constexpr int kSumRows = 16;   // threads that a column of the final sums is split over
constexpr int kSumChains = 8;  // sums of a thread (short chains: 2368 partial rows in 21 + 3 + 16 additions)

// Where the 8 * j + e-th of a thread's NV * 8 channels of a row is: with VEC, 8 consecutive channels per j (16-byte
// accesses; C % 8 == 0 and every row 16-byte aligned), else one channel per access, a warp's side by side and
// its NV * 256 channels together, so that j and e only add constants and all warps but the last have whole rows
// (an address and a bound per channel were two thirds of the instructions for odd widths).
template <bool VEC, int NV>
__device__ __forceinline__ int channel(int j, int e) {
  const int i = static_cast<int>(threadIdx.x);
  return VEC ? (j * static_cast<int>(blockDim.x) + i) * 8 + e : (i >> 5) * (NV * 256) + (i & 31) + (j * 8 + e) * 32;
}
// Whether all of a thread's channels are there (the same for a whole warp).
template <int NV>
__device__ __forceinline__ bool whole(int C) {
  return (static_cast<int>(threadIdx.x >> 5) + 1) * (NV * 256) <= C;
}

template <bool VEC, int NV, typename T>
__device__ __forceinline__ void load8(const T* row, int j, int C, float (&v)[8]) {
  const int c0 = channel<VEC, NV>(j, 0);
  if (VEC) {
    if (c0 < C) {
      Raw8<T> w;
      w.load(row + c0);
      w.unpack(v);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  } else {
    const T* const p = row + c0;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c0 + e * 32 < C ? to_f32(p[e * 32]) : 0.f;
  }
}

template <bool VEC, int NV, typename T>
__device__ __forceinline__ void store8(T* row, int j, int C, const float (&v)[8]) {
  const int c0 = channel<VEC, NV>(j, 0);
  if (VEC) {
    if (c0 < C) {
      Raw8<T> w;
      w.pack(v);
      w.store(row + c0);
    }
  } else {
    T* const p = row + c0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + e * 32 < C) p[e * 32] = from_f32<T>(v[e]);
  }
}

// Sums of N (1 or 3) values over a CTA of at most MAX_WARPS warps, the same in every thread and in a fixed order.
// `buf` (N * 32 floats, cleared by clear_sums) is one of two areas used in turn, so one barrier per call is enough.
// Three values share the rounds within a warp: after two of them a lane has the sum of only one value.
template <int MAX_WARPS, int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf) {
  static_assert(N == 1 || N == 3, "");
  constexpr int kWarps = MAX_WARPS <= 8 ? 8 : MAX_WARPS <= 16 ? 16 : 32;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  auto add = [](float x, int o) { return x + __shfl_xor_sync(0xffffffffu, x, o); };
  float z;
  int mine = 0;
  if (N == 1) {
    z = add(add(v[0], 16), 8);
  } else {
    const bool a = lane & 16, b = lane & 8;  // lanes 0-7: the first, 16-23: the second, 8-15 and 24-31: the third
    const float x = (a ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, a ? v[0] : v[1], 16), y = add(v[N - 1], 16);
    z = (b ? y : x) + __shfl_xor_sync(0xffffffffu, b ? x : y, 8);
    mine = b ? 2 : a ? 1 : 0;
  }
  z = add(add(add(z, 4), 2), 1);
  if (warps == 1) {
    if (N == 1) {
      v[0] = z;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, z, i == 0 ? 0 : i == 1 ? 16 : 8);
    }
    __syncwarp();
    return;
  }
  if (N == 1 ? lane == 0 : (lane & 7) == 0 && lane < 24) buf[mine * 32 + (threadIdx.x >> 5)] = z;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {  // four warps' sums a lane
    const float4 f = *reinterpret_cast<const float4*>(buf + i * 32 + (lane & (kWarps / 4 - 1)) * 4);
    v[i] = (f.x + f.y) + (f.z + f.w);
#pragma unroll
    for (int o = kWarps / 8; o > 0; o >>= 1) v[i] = add(v[i], o);
  }
}
// (The entries of warps that are not there; written before the first barrier of block_sums.)
template <int N>
__device__ __forceinline__ void clear_sums(float (&buf)[2][N]) {
  const int i = static_cast<int>(threadIdx.x);
  if (i < 32 && i >= static_cast<int>(blockDim.x >> 5))
#pragma unroll
    for (int k = 0; k < 2 * N; k += 32) buf[k / N][k % N + i] = 0.f;
}

// The gate row of a row that only moves on: a 64-bit division costs as much as the rest of a row's
// arithmetic, and the gate row seldom changes.
struct GateRow {
  int64_t index = -1, end = 0;
  __device__ __forceinline__ int64_t of(int64_t row, int64_t per) {
    if (row >= end) {
      index = row / per;
      end = (index + 1) * per;
    }
    return index;
  }
};

struct FwdArgs {
  const void *residual, *block, *gate;
  const float *post, *pre;
  void *residual_out, *normed;
  int64_t rows, per_gate;
  int C;
  float alpha, eps;
};

template <typename T, int NV, bool VEC, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) block_norm_fwd_kernel(const FwdArgs a) {
  __shared__ __align__(16) float sums[2][32];
  clear_sums(sums);
  const int C = a.C;
  const float inv = 1.f / static_cast<float>(C);
  GateRow gate_row;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float r[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) load8<VEC, NV>(static_cast<const T*>(a.residual) + row * C, j, C, r[j]);
    if (a.block) {
      float b[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) load8<VEC, NV>(static_cast<const T*>(a.block) + row * C, j, C, b[j]);
      if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(b[j][e], b[j][e], s[0]);
        block_sums<MAX_THREADS / 32>(s, sums[0]);
        const float bs = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float w[8];
          load8<VEC, NV>(a.post, j, C, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) b[j][e] = b[j][e] * bs * w[e];
        }
      }
      if (a.gate) {
        const T* gr = static_cast<const T*>(a.gate) + gate_row.of(row, a.per_gate) * C;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float g[8];
          load8<VEC, NV>(gr, j, C, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) b[j][e] *= g[e];
        }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = fmaf(a.alpha, b[j][e], r[j][e]);
    }
    if (a.residual_out)
#pragma unroll
      for (int j = 0; j < NV; ++j) store8<VEC, NV>(static_cast<T*>(a.residual_out) + row * C, j, C, r[j]);
    if (a.normed) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(r[j][e], r[j][e], s[0]);
      block_sums<MAX_THREADS / 32>(s, sums[1]);
      const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8];
        load8<VEC, NV>(a.pre, j, C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = r[j][e] * rs * w[e];
        store8<VEC, NV>(static_cast<T*>(a.normed) + row * C, j, C, r[j]);
      }
    }
    if (!a.post || !a.normed) __syncthreads();  // with both, the reductions' areas alternate
  }
}

struct BwdArgs {
  const void *residual_out, *block, *gate, *d_out, *d_normed;
  const float *post, *pre;
  void *d_residual, *d_block;
  float *sum_pre, *sum_post, *sum_gate;  // partial sums [ctas][C], [ctas][C], [ctas][2][C] or NULL
  float* d_gate;
  int64_t rows, per_gate, rows_per_cta;
  int C;
  float alpha, eps;
};

// One CTA per rows_per_cta consecutive rows.  The sums over rows stay with the thread that owns the
// channel (in registers where SUMS_IN_REGS, else in the CTA's own rows of the partial sums) and
// end as one row of partial sums per CTA.  A gate row's sum is written out when the CTA has seen all of
// its rows, else as the CTA's first (0: begun by an earlier CTA) or last (1) partial.
template <typename T, int NV, bool VEC, bool SUMS_IN_REGS, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) block_norm_bwd_kernel(const BwdArgs a) {
  __shared__ __align__(16) float sums[2][3 * 32];
  clear_sums(sums);
  const int C = a.C;
  const float inv = 1.f / static_cast<float>(C);
  const int64_t first = blockIdx.x * a.rows_per_cta, last = min(first + a.rows_per_cta, a.rows);
  const int64_t cta = blockIdx.x;
  float* const part_pre = a.sum_pre ? a.sum_pre + cta * C : nullptr;
  float* const part_post = a.sum_post ? a.sum_post + cta * C : nullptr;
  constexpr int KV = SUMS_IN_REGS ? NV : 1;
  float apre[KV][8], apost[KV][8], agate[KV][8];
  const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (SUMS_IN_REGS) {
#pragma unroll
    for (int j = 0; j < KV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) apre[j][e] = apost[j][e] = agate[j][e] = 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (part_pre) store8<VEC, NV>(part_pre, j, C, zero);
      if (part_post) store8<VEC, NV>(part_post, j, C, zero);
    }
  }
  float* gate_to = nullptr;  // where the current gate row's sum goes
  GateRow gate_row;
  for (int64_t row = first; row < last; ++row) {
    const bool new_gate = a.gate && row >= gate_row.end;
    const T* const g_row = a.gate ? static_cast<const T*>(a.gate) + gate_row.of(row, a.per_gate) * C : nullptr;
    if (a.sum_gate && new_gate) {
      if (SUMS_IN_REGS && gate_to) {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
          store8<VEC, NV>(gate_to, j, C, agate[j]);
#pragma unroll
          for (int e = 0; e < 8; ++e) agate[j][e] = 0.f;
        }
      }
      const int64_t g = gate_row.index, begin = g * a.per_gate, end = min(begin + a.per_gate, a.rows);
      if (begin < first) gate_to = a.sum_gate + (cta * 2) * C;
      else if (end > last) gate_to = a.sum_gate + (cta * 2 + 1) * C;
      else gate_to = a.d_gate + g * C;
      if (!SUMS_IN_REGS)
#pragma unroll
        for (int j = 0; j < NV; ++j) store8<VEC, NV>(gate_to, j, C, zero);
    }
    float dr[NV][8], b[NV][8];
    float s[3] = {0.f, 0.f, 0.f};  // r'^2, u r', b^2
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (a.block) {
        load8<VEC, NV>(static_cast<const T*>(a.block) + row * C, j, C, b[j]);
        if (a.post)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[2] = fmaf(b[j][e], b[j][e], s[2]);
      }
      if (a.d_out) {
        load8<VEC, NV>(static_cast<const T*>(a.d_out) + row * C, j, C, dr[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[j][e] = 0.f;
      }
    }
    if (a.d_normed) {
      float r[NV][8], dn[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load8<VEC, NV>(static_cast<const T*>(a.residual_out) + row * C, j, C, r[j]);
        load8<VEC, NV>(static_cast<const T*>(a.d_normed) + row * C, j, C, dn[j]);
        float w[8];
        load8<VEC, NV>(a.pre, j, C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = fmaf(r[j][e], r[j][e], s[0]);
          s[1] = fmaf(dn[j][e] * w[e], r[j][e], s[1]);
        }
      }
      block_sums<MAX_THREADS / 32>(s, sums[0]);
      const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
      const float m = s[1] * inv * rs * rs;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8], add[8];
        load8<VEC, NV>(a.pre, j, C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dr[j][e] = fmaf(rs, fmaf(dn[j][e], w[e], -r[j][e] * m), dr[j][e]);
          add[e] = dn[j][e] * r[j][e] * rs;
        }
        if (part_pre) {
          if (SUMS_IN_REGS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) apre[SUMS_IN_REGS ? j : 0][e] += add[e];
          } else {
            float t[8];
            load8<VEC, NV>(part_pre, j, C, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += add[e];
            store8<VEC, NV>(part_pre, j, C, t);
          }
        }
      }
    } else if (a.post) {
      block_sums<MAX_THREADS / 32>(s, sums[0]);
    }
    if (a.d_residual)
#pragma unroll
      for (int j = 0; j < NV; ++j) store8<VEC, NV>(static_cast<T*>(a.d_residual) + row * C, j, C, dr[j]);
    if (a.block) {
      const float bs = a.post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.f;
      float c[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8];
        if (a.post) {
          load8<VEC, NV>(a.post, j, C, w);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = 1.f;
        }
        if (a.sum_gate) {
          float add[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) add[e] = a.alpha * dr[j][e] * (b[j][e] * bs * w[e]);
          if (SUMS_IN_REGS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) agate[SUMS_IN_REGS ? j : 0][e] += add[e];
          } else {
            float t[8];
            load8<VEC, NV>(gate_to, j, C, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += add[e];
            store8<VEC, NV>(gate_to, j, C, t);
          }
        }
        float g[8];
        if (g_row) {
          load8<VEC, NV>(g_row, j, C, g);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[j][e] = a.alpha * g[e] * dr[j][e];  // q
        if (part_post) {
          float add[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) add[e] = dr[j][e] * (b[j][e] * bs);
          if (SUMS_IN_REGS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) apost[SUMS_IN_REGS ? j : 0][e] += add[e];
          } else {
            float t[8];
            load8<VEC, NV>(part_post, j, C, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += add[e];
            store8<VEC, NV>(part_post, j, C, t);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dr[j][e] *= w[e];
          c[0] = fmaf(dr[j][e], b[j][e], c[0]);
        }
      }
      float m = 0.f;
      if (a.post) {
        block_sums<MAX_THREADS / 32>(c, sums[1]);
        m = c[0] * inv * bs * bs;
      }
      if (a.d_block)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dr[j][e] = bs * (dr[j][e] - b[j][e] * m);
          store8<VEC, NV>(static_cast<T*>(a.d_block) + row * C, j, C, dr[j]);
        }
    }
    if (!a.post) __syncthreads();  // with both reductions, their areas alternate
  }
  if (SUMS_IN_REGS) {
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      if (part_pre) store8<VEC, NV>(part_pre, j, C, apre[j]);
      if (part_post) store8<VEC, NV>(part_post, j, C, apost[j]);
      if (gate_to) store8<VEC, NV>(gate_to, j, C, agate[j]);
    }
  }
}

// ---- many rows of middling width: rows come through a ring in shared memory ----
//
// Loading a row into registers and then reducing it leaves the memory idle during the reductions
// unless many CTAs take turns, and registers limit those.  Here one thread requests whole rows with bulk
// copies, as far ahead as the ring has room, and the threads read them from shared memory, the
// backward twice (once for the sums, once for the results), so that registers hold little but sums; the
// weights wait in shared memory too.
// Rows need no alignment: a copy takes the 16-byte pieces that hold the row, which then lies at
// the same offset from a 16-byte boundary as in memory.

constexpr int kRingLow = 256, kRingHigh = 8192;  // widths served
constexpr int kRingBytes = 216 * 1024;           // of an SM
constexpr int kMaxRing = 4;
constexpr int kBwdNv = 2;                        // 8-channel vectors of a thread (one: 81 us for 4096 x 4096, not 58)

// Set when a ring gave up a wait: reported, and cleared, by bconv_block_norm_sync_status.
__device__ uint32_t block_norm_error;

__device__ __forceinline__ bool ring_gave_up(const uint32_t* gave_up) {
  return *reinterpret_cast<const volatile uint32_t*>(gave_up) != 0;
}
// Copies that were issued arrive, so a wait ends.  After a second it gives up all the same: it sets the error word and
// the CTA's flag, with which no further row is requested or waited for.  (The other copies in flight are as old by
// then.)  Out of line, it costs the 16-bit backward no registers (4096 x 4096 bf16 58.1 us, 59.3 with it inline; fp32
// 88.3 and 88.1, forward 47.2 and 46.2).
__device__ __noinline__ void ring_wait_slow(uint64_t* bar, uint32_t parity, uint32_t* gave_up) {
  const uint64_t t0 = tcdev::globaltimer();
  while (!ring_gave_up(gave_up)) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
      if (tcdev::mbar_try(bar, parity)) return;
    if (tcdev::globaltimer() - t0 > tcdev::kTimeoutNs) {
      atomicOr(&block_norm_error, kErrTimeout);
      atomicExch(gave_up, 1u);
    }
  }
}
__device__ __forceinline__ void ring_wait(uint64_t* bar, uint32_t parity, uint32_t* gave_up) {
  if (!tcdev::mbar_try(bar, parity)) ring_wait_slow(bar, parity, gave_up);
}

// Bytes of a row in a stage: the 16-byte pieces that may hold it.
__host__ __device__ constexpr int ring_row(int C, int elem) { return (C * elem + 15) / 16 * 16 + 16; }

// Requests row `row` of `rows` of up to N arrays, C channels each, into the stage `to` (one thread; everyone
// has passed a barrier since the stage was last read).  Row i lies at to + i * ring_row(), plus its offset
// from a 16-byte boundary.  Pieces that reach into the rows before and after are read whole, but not beyond
// the array: at its edges plain copies fill in.
template <typename T, bool VEC, int N>
__device__ __forceinline__ void ring_request(uint64_t* full, uint8_t* to, const T* const (&src)[N], int C, int64_t row,
                                             int64_t rows) {
  const uint32_t bytes = static_cast<uint32_t>(C) * sizeof(T);
  const int pitch = ring_row(C, sizeof(T));
  if (VEC) {
    uint32_t arrays = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) arrays += src[i] != nullptr;
    tcdev::mbar_expect_tx(full, arrays * bytes);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (src[i]) tcdev::bulk_load(to + i * pitch, src[i] + row * C, bytes, full);
  } else {
    // The plain stores of an earlier request come before these copies, which may write the same places.  (A fence in the
    // branches of those stores instead: 8000 x 2001 bf16 backward 69 us, not 61.)
    tcdev::fence_proxy_async();
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (src[i]) {
        const T* p = src[i] + row * C;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), e = a + bytes, base = a & ~uintptr_t{15};
        uintptr_t lo = base, hi = (e + 15) & ~uintptr_t{15};
        if (row == 0 && lo != a) lo += 16;
        if (row + 1 == rows && hi != e) hi -= 16;
        T* const at = reinterpret_cast<T*>(to + i * pitch + (a - base));
        if (lo > a)
          for (int c = 0; reinterpret_cast<uintptr_t>(p + c) < lo; ++c) at[c] = p[c];
        if (hi < e)
          for (int c = static_cast<int>(reinterpret_cast<const T*>(hi) - p); c < C; ++c) at[c] = p[c];
        tcdev::bulk_load(to + i * pitch + (lo - base), reinterpret_cast<const void*>(lo), static_cast<uint32_t>(hi - lo), full);
        sum += static_cast<uint32_t>(hi - lo);
      }
    tcdev::mbar_expect_tx(full, sum);  // (the arrival: behind the plain copies)
  }
}

// Where array i's row lies in a stage.
template <typename T, bool VEC>
__device__ __forceinline__ const T* ring_at(const uint8_t* stage, int i, const T* src, int C, int64_t row) {
  const int shift = VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(src + row * C) & 15u);
  return reinterpret_cast<const T*>(stage + i * ring_row(C, sizeof(T)) + shift);
}

__device__ __forceinline__ void ring_init(uint64_t* full, int stages, uint32_t* gave_up) {
  if (threadIdx.x == 0) {
    *gave_up = 0;
    for (int s = 0; s < stages; ++s) tcdev::mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// Loads and stores of rows in a loop that skips a thread's vectors behind the row (`absent`: filling them with zeros,
// load by load, was a sixth of the backward's instructions); ALL: the thread's channels are all there.
template <bool VEC, int NV>
__device__ __forceinline__ bool absent(int j, int C) {
  return VEC && channel<true, NV>(j, 0) >= C;
}
template <bool VEC, bool ALL, int NV, typename T>
__device__ __forceinline__ void get8(const T* row, int j, int C, float (&v)[8]) {
  const T* const p = row + channel<VEC, NV>(j, 0);
  if (VEC) {
    Raw8<T> w;
    w.load(p);
    w.unpack(v);
  } else if (ALL) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(p[e * 32]);
  } else {
    load8<false, NV>(row, j, C, v);
  }
}
template <bool VEC, bool ALL, int NV, typename T>
__device__ __forceinline__ void put8(T* row, int j, int C, const float (&v)[8]) {
  T* const p = row + channel<VEC, NV>(j, 0);
  if (VEC) {
    Raw8<T> w;
    w.pack(v);
    w.store(p);
  } else if (ALL) {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e * 32] = from_f32<T>(v[e]);
  } else {
    store8<false, NV>(row, j, C, v);
  }
}
// The same as pairs, for the packed arithmetic.
template <bool VEC, bool ALL, int NV, typename T>
__device__ __forceinline__ void get4x2(const T* row, int j, int C, uint64_t (&v)[4]) {
  float f[8];
  get8<VEC, ALL, NV>(row, j, C, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <bool VEC, bool ALL, int NV, typename T>
__device__ __forceinline__ void put4x2(T* row, int j, int C, const uint64_t (&v)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = half_of(v[i / 2], i & 1);
  put8<VEC, ALL, NV>(row, j, C, f);
}
__device__ __forceinline__ float both(uint64_t v) { return half_of(v, 0) + half_of(v, 1); }
// f(std::true_type) for threads whose channels are all there, else f(std::false_type); the same for a warp.
template <bool VEC, typename F>
__device__ __forceinline__ void with_channels(bool all, F&& f) {
  if (VEC || all) f(std::true_type{});
  else f(std::false_type{});
}

// Weights of a thread's channels in shared memory, read and written by that thread alone (so without barriers):
// vector j's eight as two float4, side by side over the threads.
struct OwnWeights {
  float4* at;
  __device__ __forceinline__ void put(int j, const float (&w)[8]) {
    at[(2 * j) * blockDim.x + threadIdx.x] = make_float4(w[0], w[1], w[2], w[3]);
    at[(2 * j + 1) * blockDim.x + threadIdx.x] = make_float4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void get(int j, uint64_t (&w)[4]) const {
    const float4 a = at[(2 * j) * blockDim.x + threadIdx.x], b = at[(2 * j + 1) * blockDim.x + threadIdx.x];
    w[0] = pair(a.x, a.y); w[1] = pair(a.z, a.w);
    w[2] = pair(b.x, b.y); w[3] = pair(b.z, b.w);
  }
};
// Two sets of them lie in front of the ring.
__host__ __device__ constexpr int own_weight_bytes(int threads, int nv) { return threads * nv * 8 * 4; }

// alpha * gate * post of this thread's channels (either may be NULL: 1)
template <typename T, bool VEC, int NV>
__device__ __forceinline__ void put_gate_post(OwnWeights W, float alpha, const T* gate, const float* post, int C) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float g[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = w[e] = 1.f;
    if (gate) load8<VEC, NV>(gate, j, C, g);
    if (post) load8<VEC, NV>(post, j, C, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= alpha * g[e];
    W.put(j, w);
  }
}

// NV: 8-channel vectors of a thread.  Two, or one for fp32, whose rows leave room for only half as many CTAs (4096 x 4096:
// 46.4 us against 50.1, 8000 x 2001: 50.3 against 60.6; bf16 30.1 against 28.5).
template <typename T, bool VEC, int NV, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, MAX_THREADS == 256                                      ? 3
                                               : MAX_THREADS == 384 || (NV == 1 && MAX_THREADS == 512) ? 2
                                                                                                       : 1)
    block_norm_fwd_ring_kernel(const FwdArgs a, int stages) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sums[2][32];
  __shared__ uint64_t full[kMaxRing];
  __shared__ uint32_t gave_up;
  clear_sums(sums);
  const bool all = whole<NV>(a.C);
  const int C = a.C, stage_bytes = 2 * ring_row(C, sizeof(T)), own = own_weight_bytes(blockDim.x, NV);
  OwnWeights pre{reinterpret_cast<float4*>(smem)}, gate_post{reinterpret_cast<float4*>(smem + own)};
  uint8_t* const ring = smem + 2 * own;
  const float inv = 1.f / static_cast<float>(C);
  ring_init(full, stages, &gave_up);
  const int64_t step = gridDim.x;
  const T* const src[2] = {static_cast<const T*>(a.residual), static_cast<const T*>(a.block)};
  if (threadIdx.x < 32 && tcdev::elect_one())
    for (int i = 0; i < stages && blockIdx.x + i * step < a.rows; ++i)
      ring_request<T, VEC>(&full[i], ring + i * stage_bytes, src, C, blockIdx.x + i * step, a.rows);
  __syncwarp();
  if (a.pre)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[8];
      load8<VEC, NV>(a.pre, j, C, w);
      pre.put(j, w);
    }
  if (!a.gate) put_gate_post<T, VEC, NV>(gate_post, a.alpha, nullptr, a.post, C);
  int s = 0;
  uint32_t parity = 0;
  GateRow gate_row;
  for (int64_t row = blockIdx.x; row < a.rows; row += step) {
    if (a.gate && row >= gate_row.end)
      put_gate_post<T, VEC, NV>(gate_post, a.alpha, static_cast<const T*>(a.gate) + gate_row.of(row, a.per_gate) * C, a.post, C);
    ring_wait(&full[s], parity, &gave_up);
    uint8_t* const stage = ring + s * stage_bytes;
    const T *const r_row = ring_at<T, VEC>(stage, 0, src[0], C, row), *const b_row = ring_at<T, VEC>(stage, 1, src[1], C, row);
    uint64_t r[NV][4], b[NV][4], qq = 0;
    with_channels<VEC>(all, [&](auto is_all) {
      constexpr bool ALL = decltype(is_all)::value;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (absent<VEC, NV>(j, C)) continue;
        get4x2<VEC, ALL, NV>(r_row, j, C, r[j]);
        if (a.block) {
          get4x2<VEC, ALL, NV>(b_row, j, C, b[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) qq = fma2(b[j][i], b[j][i], qq);
        }
      }
    });
    float q[1] = {both(qq)};
    if (a.post) block_sums<MAX_THREADS / 32>(q, sums[0]);
    else __syncthreads();
    if (threadIdx.x < 32 && row + stages * step < a.rows && tcdev::elect_one() && !ring_gave_up(&gave_up))  // everyone has read this stage
      ring_request<T, VEC>(&full[s], stage, src, C, row + stages * step, a.rows);
    __syncwarp();
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
    if (a.block) {
      const float bs = a.post ? rsqrtf(fmaf(q[0], inv, a.eps)) : 1.f;
      const uint64_t bs2 = pair(bs, bs);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (absent<VEC, NV>(j, C)) continue;
        uint64_t w[4];
        gate_post.get(j, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[j][i] = fma2(mul2(b[j][i], bs2), w[i], r[j][i]);
      }
    }
    uint64_t tt = 0;
    with_channels<VEC>(all, [&](auto is_all) {
      constexpr bool ALL = decltype(is_all)::value;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (absent<VEC, NV>(j, C)) continue;
        if (a.residual_out) put4x2<VEC, ALL, NV>(static_cast<T*>(a.residual_out) + row * C, j, C, r[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tt = fma2(r[j][i], r[j][i], tt);
      }
    });
    if (a.normed) {
      float t[1] = {both(tt)};
      block_sums<MAX_THREADS / 32>(t, sums[1]);
      const float rs = rsqrtf(fmaf(t[0], inv, a.eps));
      const uint64_t rs2 = pair(rs, rs);
      with_channels<VEC>(all, [&](auto is_all) {
        constexpr bool ALL = decltype(is_all)::value;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (absent<VEC, NV>(j, C)) continue;
          uint64_t w[4];
          pre.get(j, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = mul2(mul2(r[j][i], rs2), w[i]);
          put4x2<VEC, ALL, NV>(static_cast<T*>(a.normed) + row * C, j, C, w);
        }
      });
    }
    if (a.post && !a.normed) __syncthreads();  // (otherwise there are two barriers a row, and the areas alternate)
  }
}

// As block_norm_bwd_kernel.  While the gate stays the same, d_post_weight and d_gate are one sum
//     S = sum_rows a dR b bs     d_gate = w_post S     d_post_weight = g S
// times what does not change, so registers hold S, and d_post_weight's partial sums (in memory) are brought up
// to date with the gate.  A row's stage is requested again in the next row, behind the barrier that shows that
// everyone is done with it (all but the block's row already behind the row's second sum: 4096 x 4096 bf16 58.9 us
// against 58.5, fp32 85.5 against 88.1).
template <typename T, bool VEC, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS, MAX_THREADS == 256 ? 2 : 1) block_norm_bwd_ring_kernel(const BwdArgs a, int stages) {
  constexpr int NV = kBwdNv;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float sums[2][3 * 32];
  __shared__ uint64_t full[kMaxRing];
  __shared__ uint32_t gave_up;
  clear_sums(sums);
  const bool all = whole<NV>(a.C);
  const int C = a.C, stage_bytes = 4 * ring_row(C, sizeof(T)), own = own_weight_bytes(blockDim.x, NV);
  OwnWeights pre{reinterpret_cast<float4*>(smem)}, gate_post{reinterpret_cast<float4*>(smem + own)};
  uint8_t* const ring = smem + 2 * own;
  const float inv = 1.f / static_cast<float>(C);
  const int64_t first = blockIdx.x * a.rows_per_cta, last = min(first + a.rows_per_cta, a.rows), cta = blockIdx.x;
  ring_init(full, stages, &gave_up);
  const T* const src[4] = {a.d_normed ? static_cast<const T*>(a.residual_out) : nullptr,
                           static_cast<const T*>(a.d_normed), static_cast<const T*>(a.d_out),
                           static_cast<const T*>(a.block)};
  if (threadIdx.x < 32 && tcdev::elect_one())
    for (int i = 0; i < stages && first + i < last; ++i)
      ring_request<T, VEC>(&full[i], ring + i * stage_bytes, src, C, first + i, a.rows);
  __syncwarp();
  if (a.pre)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[8];
      load8<VEC, NV>(a.pre, j, C, w);
      pre.put(j, w);
    }
  if (!a.gate) put_gate_post<T, VEC, NV>(gate_post, a.alpha, nullptr, a.post, C);
  uint64_t apre[NV][4], sum[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) apre[j][i] = sum[j][i] = 0;
  // the sum of the rows of one gate row goes where it belongs
  float* gate_to = nullptr;
  GateRow gate_row;
  const T* g_row = nullptr;
  bool flushed = false;
  auto flush = [&]() {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8], w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = half_of(sum[j][e / 2], e & 1);
      if (gate_to) {
        if (a.post) load8<VEC, NV>(a.post, j, C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = a.post ? w[e] * f[e] : f[e];
        store8<VEC, NV>(gate_to, j, C, w);
      }
      if (a.sum_post) {
        float t[8];
        if (g_row) load8<VEC, NV>(g_row, j, C, w);
        if (flushed) load8<VEC, NV>(a.sum_post + cta * C, j, C, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float add = g_row ? w[e] * f[e] : f[e];
          t[e] = flushed ? t[e] + add : add;
        }
        store8<VEC, NV>(a.sum_post + cta * C, j, C, t);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[j][i] = 0;
    }
    flushed = true;
  };
  int s = 0;
  uint32_t parity = 0;
  for (int64_t row = first; row < last; ++row) {
    if (a.gate && row >= gate_row.end) {
      if (g_row) flush();
      const int64_t g = gate_row.of(row, a.per_gate), begin = g * a.per_gate;
      g_row = static_cast<const T*>(a.gate) + g * C;
      put_gate_post<T, VEC, NV>(gate_post, a.alpha, g_row, a.post, C);
      if (a.sum_gate) {
        if (begin < first) gate_to = a.sum_gate + (cta * 2) * C;
        else if (min(gate_row.end, a.rows) > last) gate_to = a.sum_gate + (cta * 2 + 1) * C;
        else gate_to = a.d_gate + g * C;
      }
    }
    ring_wait(&full[s], parity, &gave_up);
    uint8_t* const stage = ring + s * stage_bytes;
    const T *const r_row = ring_at<T, VEC>(stage, 0, src[0], C, row), *const dn_row = ring_at<T, VEC>(stage, 1, src[1], C, row),
            *const do_row = ring_at<T, VEC>(stage, 2, src[2], C, row), *const b_row = ring_at<T, VEC>(stage, 3, src[3], C, row);
    uint64_t tr = 0, tu = 0, tb = 0;  // r'^2, u r', b^2
    with_channels<VEC>(all, [&](auto is_all) {
      constexpr bool ALL = decltype(is_all)::value;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (absent<VEC, NV>(j, C)) continue;
        if (a.d_normed) {
          uint64_t r[4], dn[4], w[4];
          get4x2<VEC, ALL, NV>(r_row, j, C, r);
          get4x2<VEC, ALL, NV>(dn_row, j, C, dn);
          pre.get(j, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tr = fma2(r[i], r[i], tr);
            tu = fma2(mul2(dn[i], w[i]), r[i], tu);
          }
        }
        if (a.post) {
          uint64_t b[4];
          get4x2<VEC, ALL, NV>(b_row, j, C, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) tb = fma2(b[i], b[i], tb);
        }
      }
    });
    float t[3] = {both(tr), both(tu), both(tb)};
    block_sums<MAX_THREADS / 32>(t, sums[0]);
    const int64_t next = row - 1 + stages;
    if (threadIdx.x < 32 && row > first && next < last && tcdev::elect_one() && !ring_gave_up(&gave_up)) {
      const int sp = s == 0 ? stages - 1 : s - 1;
      ring_request<T, VEC>(&full[sp], ring + sp * stage_bytes, src, C, next, a.rows);
    }
    __syncwarp();
    const float rs = rsqrtf(fmaf(t[0], inv, a.eps)), m = t[1] * inv * rs * rs;
    const float bs = a.post ? rsqrtf(fmaf(t[2], inv, a.eps)) : 1.f, abs_ = a.alpha * bs;
    const uint64_t rs2 = pair(rs, rs), m2 = pair(-m, -m), abs2 = pair(abs_, abs_);
    uint64_t cc = 0, v[NV][4];
    with_channels<VEC>(all, [&](auto is_all) {
      constexpr bool ALL = decltype(is_all)::value;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (absent<VEC, NV>(j, C)) continue;
        uint64_t dr[4], w[4];
        if (a.d_out) {
          get4x2<VEC, ALL, NV>(do_row, j, C, dr);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) dr[i] = 0;
        }
        if (a.d_normed) {
          uint64_t r[4], dn[4];
          get4x2<VEC, ALL, NV>(r_row, j, C, r);
          get4x2<VEC, ALL, NV>(dn_row, j, C, dn);
          pre.get(j, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dr[i] = fma2(rs2, fma2(dn[i], w[i], mul2(r[i], m2)), dr[i]);
            apre[j][i] = fma2(dn[i], mul2(r[i], rs2), apre[j][i]);
          }
        }
        if (a.d_residual) put4x2<VEC, ALL, NV>(static_cast<T*>(a.d_residual) + row * C, j, C, dr);
        if (a.block) {
          uint64_t b[4];
          get4x2<VEC, ALL, NV>(b_row, j, C, b);
          gate_post.get(j, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[j][i] = fma2(dr[i], mul2(b[i], abs2), sum[j][i]);
            v[j][i] = mul2(dr[i], w[i]);
            cc = fma2(v[j][i], b[i], cc);
          }
        }
      }
    });
    if (a.block) {
      float mb = 0.f;
      if (a.post) {
        float c[1] = {both(cc)};
        block_sums<MAX_THREADS / 32>(c, sums[1]);
        mb = c[0] * inv * bs * bs;
      }
      if (a.d_block) {
        const uint64_t bs2 = pair(bs, bs), mb2 = pair(-mb, -mb);
        with_channels<VEC>(all, [&](auto is_all) {
          constexpr bool ALL = decltype(is_all)::value;
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (absent<VEC, NV>(j, C)) continue;
            uint64_t b[4];
            get4x2<VEC, ALL, NV>(b_row, j, C, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = mul2(bs2, fma2(b[i], mb2, v[j][i]));
            put4x2<VEC, ALL, NV>(static_cast<T*>(a.d_block) + row * C, j, C, b);
          }
        });
      }
    }
    if (!a.block || !a.post) __syncthreads();  // with both reductions, their areas alternate
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
  allow_next_grid();
  flush();
  if (a.sum_pre)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = half_of(apre[j][e / 2], e & 1);
      store8<VEC, NV>(a.sum_pre + cta * C, j, C, f);
    }
}

struct SumArgs {
  const float *sum_pre, *sum_post, *sum_gate;
  float *d_pre, *d_post, *d_gate;
  int64_t rows, per_gate, rows_per_cta;
  int C, ctas, by_gate;
};

// The partial rows of 32 channels, added in a fixed order.  blockIdx.y: 0 d_pre, 1 d_post, above that the gate
// rows that several CTAs share: by the gate row (2 + g), or, with more gate rows than CTAs, by the CTA i that
// found it begun and is the first to do so (1 + i).
__global__ void block_norm_sum_kernel(const SumArgs a) {
  __shared__ float part[kSumRows][33];
  wait_prior_grid();
  const int c = blockIdx.x * 32 + threadIdx.x, y = blockIdx.y;
  const float* from = nullptr;  // row of partial `from_first`
  float* to = nullptr;
  int64_t n = a.ctas, step = a.C;
  const float* extra = nullptr;  // the partial that comes before them
  if (y == 0) {
    from = a.sum_pre;
    to = a.d_pre;
  } else if (y == 1) {
    from = a.sum_post;
    to = a.d_post;
  } else if (a.d_gate) {
    int64_t g = y - 2, i;
    if (a.by_gate) {
      i = g * a.per_gate / a.rows_per_cta + 1;
    } else {
      i = y - 1;
      g = i * a.rows_per_cta / a.per_gate;
    }
    const int64_t begin = g * a.per_gate, end = min(begin + a.per_gate, a.rows), start = i * a.rows_per_cta;
    if (begin >= start || begin / a.rows_per_cta + 1 != i || end <= start) return;
    step = 2 * static_cast<int64_t>(a.C);
    from = a.sum_gate + i * step;
    extra = a.sum_gate + (i - 1) * step + a.C;
    n = (end - 1) / a.rows_per_cta - i + 1;
    to = a.d_gate + g * a.C;
  }
  if (!to) return;
  float s = 0.f;
  if (c < a.C) {
    float t[kSumChains] = {};
    const float* p = from + threadIdx.y * step + c;
    step *= kSumRows;
    int left = (static_cast<int>(n) - static_cast<int>(threadIdx.y) + kSumRows - 1) / kSumRows;
    for (; left >= kSumChains; left -= kSumChains)
#pragma unroll
      for (int k = 0; k < kSumChains; ++k, p += step) t[k] += *p;
    if (left >= kSumChains / 2) {
#pragma unroll
      for (int k = 0; k < kSumChains / 2; ++k, p += step) t[k] += *p;
      left -= kSumChains / 2;
    }
#pragma unroll 1
    for (; left > 0; --left, p += step) t[kSumChains - 1] += *p;
#pragma unroll
    for (int w = kSumChains / 2; w > 0; w /= 2)
#pragma unroll
      for (int k = 0; k < w; ++k) t[k] += t[k + w];
    s = extra && threadIdx.y == 0 ? extra[c] + t[0] : t[0];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.C) {
    for (int i = 1; i < kSumRows; ++i) s += part[i][threadIdx.x];
    to[c] = s;
  }
}

struct Shape {
  int threads, nv;
};

// Threads and 8-channel vectors per thread of one row.
Shape shape_for(int C, int max_nv) {
  const int vecs = (C + 7) / 8;
  int nv = 1;
  while (nv < max_nv && vecs > 256 * nv) nv *= 2;
  return {std::min(1024, round_up((vecs + nv - 1) / nv, 32)), nv};
}

// A ring kernel's threads, stages of `stage` bytes and CTAs per SM, of at most `ctas` (what its registers allow),
// and the bytes of shared memory of a CTA.  All of these CTAs have to be resident, since each gets its share of the
// rows: a CTA's static shared memory (below 1 KB) and the 1 KB that the hardware keeps for it count as well, which for
// narrow rows is much of the SM's 228 KB.  (30000 x 384 bf16 backward with 16 CTAs planned and 15 resident: 70 us.)
struct Ring {
  int threads, stages, ctas, bytes;
};
constexpr int kSmBytes = 228 * 1024, kCtaBytes = 2 * 1024;
// Threads, in whole warps, for C channels in vectors of 8, nv of them a thread.
constexpr int ring_threads(int C, int nv) { return (C + 8 * nv * 32 - 1) / (8 * nv * 32) * 32; }
constexpr Ring ring_for(int C, int nv, int stage, int ctas) {
  Ring r{};
  r.threads = ring_threads(C, nv);
  const int own = 2 * own_weight_bytes(r.threads, nv), least = own + 2 * stage;
  r.ctas = std::max(1, std::min({ctas, kRingBytes / least, kSmBytes / (least + kCtaBytes)}));
  const int room = std::min(kRingBytes / r.ctas, kSmBytes / r.ctas - kCtaBytes);
  r.stages = std::max(2, std::min(kMaxRing, (room - own) / stage));
  r.bytes = own + r.stages * stage;
  return r;
}
constexpr Ring fwd_ring(int C, int elem) {
  const int nv = elem == 4 ? 1 : 2, threads = ring_threads(C, nv);
  const int ctas = nv == 1 ? 2 * 512 / threads : threads <= 256 ? 3 * 256 / threads : threads <= 384 ? 2 : 1;
  return ring_for(C, nv, 2 * ring_row(C, elem), ctas);
}
constexpr Ring bwd_ring(int C, int elem) {
  return ring_for(C, kBwdNv, 4 * ring_row(C, elem), C <= 4096 ? 2 * 256 / ring_threads(C, kBwdNv) : 1);
}
constexpr bool resident(const Ring& r) { return r.bytes > kRingBytes || r.ctas * (r.bytes + kCtaBytes) <= kSmBytes; }
constexpr bool all_resident(int first, int last) {
  for (int C = first; C <= last; ++C)
    for (int elem = 2; elem <= 4; elem += 2)
      if (!resident(fwd_ring(C, elem)) || !resident(bwd_ring(C, elem))) return false;
  return true;
}
template <int I>
constexpr bool kResident = all_resident(64 * I + 1, 64 * I + 64);  // (in parts: one expression may only be so long)
template <int... I>
constexpr bool every_resident(std::integer_sequence<int, I...>) {
  return (kResident<I + kRingLow / 64> && ...);
}
static_assert(every_resident(std::make_integer_sequence<int, (kRingHigh - kRingLow) / 64>()),
              "every planned CTA has its shared memory");

// Whether a ring of rows of this width has room (two stages fit).
bool ring_serves(int C, const Ring& r) { return C > kRingLow && C <= kRingHigh && r.bytes <= kRingBytes; }

// Whether there is enough to request ahead: below that the plain kernels start sooner.  Measured with rows in L2, ring
// against plain: forward bf16 2000 x 2000 8.4 us against 8.2, 1200 x 4000 9.1 against 10.9, fp32 600 x 4000 11.1 against 10.8,
// 1200 x 4000 17 against 20; backward bf16 450 x 2000 15.1 against 13.9, 600 x 2000 14.3 against 15.6, bf16
// 1200 x 2001 23.3 against 23.0, fp32 1200 x 2000 23.4 against 21.8, 2000 x 2000 28.9 against 31.8.
bool fwd_ring_pays(int64_t rows, int C, int elem) {
  const int64_t sms = current_sm_count();
  return rows > 2 * sms && rows * C * elem >= 65536 * sms;
}
bool bwd_ring_pays(int64_t rows, int C, int elem, bool vec) {
  const int64_t sms = current_sm_count();
  return rows > 2 * sms && rows * C >= (vec && elem == 2 ? 8192 : 16384) * sms;
}

int64_t bwd_ctas(const bconv_block_norm_desc_t* d, int64_t* rows_per_cta) {
  const int elem = dtype_bytes(d->dtype);
  // (rows of one warp: 16 CTAs an SM, 16000 x 111 bf16 in 25 us, 167 with two)
  const Ring r = bwd_ring(d->width, elem);
  const int per_sm = ring_serves(d->width, r) ? r.ctas : d->width <= kRingLow ? 16 : 2;
  const int64_t most = static_cast<int64_t>(current_sm_count()) * per_sm;
  const int64_t per = std::max<int64_t>(1, ceil_div(d->rows, most));
  if (rows_per_cta) *rows_per_cta = per;
  return d->rows > 0 ? ceil_div(d->rows, per) : 0;
}

bconv_status_t check_desc(const bconv_block_norm_desc_t* d) {
  if (!d || d->rows < 0 || d->rows > (int64_t{1} << 40) || d->width < 1 || !valid_dtype(d->dtype) ||
      !(d->eps >= 0.f) || d->residual_scale != d->residual_scale)
    return BCONV_ERR_INVALID_ARG;
  return d->width > kMaxWidth ? BCONV_ERR_UNSUPPORTED : BCONV_OK;
}

// Rows that share a gate row: no more than there are (sums with larger numbers could overflow).
int64_t per_gate(const bconv_block_norm_desc_t* d, const void* gate) {
  return gate ? std::min(d->rows_per_gate, d->rows) : 1;
}

bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

bool all_elem(std::initializer_list<const void*> ps, int t) {
  for (const void* p : ps)
    if (!aligned_elem(p, t)) return false;
  return true;
}

template <typename T, int NV, bool VEC, int MAX_THREADS>
cudaError_t launch_fwd(const FwdArgs& a, int threads, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(current_sm_count()) * std::max(1, 1024 / threads);
  block_norm_fwd_kernel<T, NV, VEC, MAX_THREADS><<<static_cast<unsigned>(std::min(a.rows, most)), threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int NV, bool VEC, int MAX_THREADS>
cudaError_t launch_bwd(const BwdArgs& a, int64_t ctas, int threads, cudaStream_t s) {
  block_norm_bwd_kernel<T, NV, VEC, NV <= 2, MAX_THREADS><<<static_cast<unsigned>(ctas), threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <auto Kern, typename Args>
cudaError_t launch_ring(const Args& a, int64_t ctas, const Ring& r, cudaStream_t s) {
  const cudaError_t e = allow_smem<Kern>(kRingBytes);
  if (e != cudaSuccess) return e;
  Kern<<<static_cast<unsigned>(ctas), r.threads, r.bytes, s>>>(a, r.stages);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch_fwd_ring(const FwdArgs& a, cudaStream_t s) {
  constexpr int kNv = sizeof(T) == 4 ? 1 : 2, kFew = 512 / kNv;
  const Ring r = fwd_ring(a.C, sizeof(T));
  const int64_t ctas = std::min(a.rows, static_cast<int64_t>(current_sm_count()) * r.ctas);
  if (r.threads <= kFew) return launch_ring<block_norm_fwd_ring_kernel<T, VEC, kNv, kFew>>(a, ctas, r, s);
  if constexpr (kNv == 2)  // (8000 x 4099 bf16: 72 us, 100 with one CTA an SM; 6000 x 6144: 50, 60)
    if (r.threads <= 384) return launch_ring<block_norm_fwd_ring_kernel<T, VEC, kNv, 384>>(a, ctas, r, s);
  return launch_ring<block_norm_fwd_ring_kernel<T, VEC, kNv, 2 * kFew>>(a, ctas, r, s);
}

template <typename T, bool VEC>
cudaError_t launch_bwd_ring(const BwdArgs& a, int64_t ctas, cudaStream_t s) {
  const Ring r = bwd_ring(a.C, sizeof(T));
  if (r.threads <= 256) return launch_ring<block_norm_bwd_ring_kernel<T, VEC, 256>>(a, ctas, r, s);
  return launch_ring<block_norm_bwd_ring_kernel<T, VEC, 512>>(a, ctas, r, s);
}

// Calls f.operator()<T, NV, VEC, MAX_THREADS> for a row shape.  The bound on the threads is what a CTA's registers are
// shared out by; the compiler does not use all of them: the backward's instances of 512 threads (8193 to 16384 channels)
// spill up to 370 bytes of 128 registers, those of 1024 (wider rows) get 32 registers and spill 1.4 to 2.4 KB (2000 x
// 16384 bf16 218 us, 1000 x 32768 617).
template <typename T, typename F>
cudaError_t with_shape(const Shape& sh, bool vec, F&& f) {
  auto pick = [&](auto nv, auto most) {
    constexpr int kNv = decltype(nv)::value, kMost = decltype(most)::value;
    return vec ? f.template operator()<T, kNv, true, kMost>() : f.template operator()<T, kNv, false, kMost>();
  };
  if (sh.nv == 1) return pick(std::integral_constant<int, 1>{}, std::integral_constant<int, 256>{});
  if (sh.nv == 2) return pick(std::integral_constant<int, 2>{}, std::integral_constant<int, 256>{});
  if (sh.threads <= 256) return pick(std::integral_constant<int, 4>{}, std::integral_constant<int, 256>{});
  if (sh.threads <= 512) return pick(std::integral_constant<int, 4>{}, std::integral_constant<int, 512>{});
  return pick(std::integral_constant<int, 4>{}, std::integral_constant<int, 1024>{});
}

struct RunFwd {
  const FwdArgs& a;
  int threads;
  cudaStream_t s;
  template <typename T, int NV, bool VEC, int MAX_THREADS>
  cudaError_t operator()() const { return launch_fwd<T, NV, VEC, MAX_THREADS>(a, threads, s); }
};

struct RunBwd {
  const BwdArgs& a;
  int64_t ctas;
  int threads;
  cudaStream_t s;
  template <typename T, int NV, bool VEC, int MAX_THREADS>
  cudaError_t operator()() const { return launch_bwd<T, NV, VEC, MAX_THREADS>(a, ctas, threads, s); }
};

}  // namespace
}  // namespace bconv

using namespace bconv;

extern "C" {

bconv_status_t bconv_block_norm_forward(const bconv_block_norm_desc_t* d, const void* residual, const void* block,
                                        const void* gate, const float* post_weight, const float* pre_weight,
                                        void* residual_out, void* normed, struct CUstream_st* stream) {
  const bconv_status_t st = check_desc(d);
  if (st != BCONV_OK || d->rows == 0) return st;
  if ((pre_weight != nullptr) != (normed != nullptr) || (!block && (gate || post_weight)) ||
      (gate && d->rows_per_gate < 1) || (!normed && !residual_out) || (block && !residual_out))
    return BCONV_ERR_INVALID_ARG;
  if (!all_elem({residual, block, gate, residual_out, normed}, d->dtype) ||
      !all_elem({post_weight, pre_weight}, BCONV_DTYPE_F32))
    return BCONV_ERR_INVALID_ARG;
  if (!residual) return BCONV_ERR_INVALID_ARG;
  FwdArgs a{residual, block, gate, post_weight, pre_weight, residual_out, normed,
            d->rows,  per_gate(d, gate), d->width, d->residual_scale, d->eps};
  const bool vec = d->width % 8 == 0 &&
                   all_aligned16({residual, block, gate, post_weight, pre_weight, residual_out, normed});
  const int elem = dtype_bytes(d->dtype);
  if (fwd_ring_pays(d->rows, d->width, elem) && ring_serves(d->width, fwd_ring(d->width, elem)))
    return from_cuda(with_dtype(d->dtype, [&](auto t) {
      using T = decltype(t);
      return vec ? launch_fwd_ring<T, true>(a, stream) : launch_fwd_ring<T, false>(a, stream);
    }));
  const Shape sh = shape_for(d->width, 4);
  return from_cuda(with_dtype(
      d->dtype, [&](auto t) { return with_shape<decltype(t)>(sh, vec, RunFwd{a, sh.threads, stream}); }));
}

int64_t bconv_block_norm_workspace_bytes(const bconv_block_norm_desc_t* d) {
  if (check_desc(d) != BCONV_OK) return -1;
  return bwd_ctas(d, nullptr) * d->width * 4 * static_cast<int64_t>(sizeof(float));
}

bconv_status_t bconv_block_norm_backward(const bconv_block_norm_desc_t* d, const void* residual_out,
                                         const void* block, const void* gate, const float* post_weight,
                                         const float* pre_weight, const void* d_residual_out, const void* d_normed,
                                         void* d_residual, void* d_block, float* d_pre_weight, float* d_post_weight,
                                         float* d_gate, void* workspace, struct CUstream_st* stream) {
  const bconv_status_t st = check_desc(d);
  if (st != BCONV_OK) return st;
  const size_t row_bytes = static_cast<size_t>(d->width) * sizeof(float);
  if (d->rows == 0) {  // (empty operands may have no address)
    cudaError_t z = d_pre_weight ? cudaMemsetAsync(d_pre_weight, 0, row_bytes, stream) : cudaSuccess;
    if (z == cudaSuccess && d_post_weight) z = cudaMemsetAsync(d_post_weight, 0, row_bytes, stream);
    return from_cuda(z);
  }
  const bool sums = d_pre_weight || d_post_weight || d_gate;
  if ((!block && (gate || post_weight || d_block)) || (gate && d->rows_per_gate < 1) ||
      (d_normed && (!pre_weight || !residual_out)) || (d_pre_weight && !pre_weight) || (d_post_weight && !post_weight) ||
      (d_gate && !gate) || (sums && !workspace))
    return BCONV_ERR_INVALID_ARG;
  if (!all_elem({residual_out, block, gate, d_residual_out, d_normed, d_residual, d_block}, d->dtype) ||
      !all_elem({post_weight, pre_weight, d_pre_weight, d_post_weight, d_gate}, BCONV_DTYPE_F32) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BCONV_ERR_INVALID_ARG;
  cudaError_t e = cudaSuccess;
  if (d_pre_weight && !d_normed) e = cudaMemsetAsync(d_pre_weight, 0, row_bytes, stream);
  if (e != cudaSuccess) return from_cuda(e);
  int64_t rows_per_cta = 0;
  const int64_t ctas = bwd_ctas(d, &rows_per_cta);
  float* ws = static_cast<float*>(workspace);
  const int64_t part = ctas * d->width;
  BwdArgs a{};
  a.residual_out = residual_out; a.block = block; a.gate = gate; a.d_out = d_residual_out; a.d_normed = d_normed;
  a.post = post_weight; a.pre = pre_weight; a.d_residual = d_residual; a.d_block = d_block;
  a.sum_pre = d_pre_weight && d_normed ? ws : nullptr;
  a.sum_post = d_post_weight ? ws + part : nullptr;
  a.sum_gate = d_gate ? ws + 2 * part : nullptr;
  a.d_gate = d_gate;
  a.rows = d->rows; a.per_gate = per_gate(d, gate); a.rows_per_cta = rows_per_cta;
  a.C = d->width; a.alpha = d->residual_scale; a.eps = d->eps;
  const bool vec = d->width % 8 == 0 && all_aligned16({residual_out, block, gate, d_residual_out, d_normed, post_weight,
                                                       pre_weight, d_residual, d_block, d_gate, workspace});
  const Shape sh = shape_for(d->width, 4);
  const int elem = dtype_bytes(d->dtype);
  const bool ring = bwd_ring_pays(d->rows, d->width, elem, vec) && ring_serves(d->width, bwd_ring(d->width, elem));
  e = with_dtype(d->dtype, [&](auto t) {
    using T = decltype(t);
    if (ring) return vec ? launch_bwd_ring<T, true>(a, ctas, stream) : launch_bwd_ring<T, false>(a, ctas, stream);
    return with_shape<T>(sh, vec, RunBwd{a, ctas, sh.threads, stream});
  });
  if (e != cudaSuccess || !sums) return from_cuda(e);
  SumArgs f{};
  f.sum_pre = a.sum_pre; f.sum_post = a.sum_post; f.sum_gate = a.sum_gate;
  f.d_pre = a.sum_pre ? d_pre_weight : nullptr; f.d_post = d_post_weight; f.d_gate = d_gate;
  f.rows = a.rows; f.per_gate = a.per_gate; f.rows_per_cta = rows_per_cta; f.C = a.C; f.ctas = static_cast<int>(ctas);
  const int64_t gates = d_gate ? ceil_div(a.rows, a.per_gate) : 0;
  f.by_gate = gates < ctas;
  const unsigned ys = static_cast<unsigned>(2 + (f.by_gate ? gates : ctas - 1));
  return from_cuda(launch_overlapped(block_norm_sum_kernel, dim3(static_cast<unsigned>(ceil_div(a.C, 32)), ys), dim3(32, kSumRows),
                                     0, stream, f));
}

bconv_status_t bconv_block_norm_sync_status(struct CUstream_st* stream) {
  uint32_t err = 0;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&err, block_norm_error, sizeof(err));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return from_cuda(e);
  }
  if (!err) return BCONV_OK;
  const uint32_t none = 0;
  e = cudaMemcpyToSymbol(block_norm_error, &none, sizeof(none));
  return e != cudaSuccess ? from_cuda(e) : err & kErrTimeout ? BCONV_ERR_TIMEOUT : BCONV_ERR_CUDA;
}

}  // extern "C"
