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
// Bound by HBM: the forward reads two and writes two arrays of rows x C, the backward reads four
// and writes two; everything between stays in registers.  One CTA holds a whole row (its threads
// 8 channels at a time), so each of the row sums is one block reduction, and the CTA walks over
// rows with the weights in registers: fp32 weights re-read per row would be as many L2 bytes as
// a bf16 row itself.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "dtype.cuh"
#include "host_util.cuh"

namespace bconv {
namespace {

constexpr int kMaxWidth = 32768;
constexpr int kSumRows = 16;  // partial rows a column of the final sums is split over

// Where a thread's 8 * j + e-th channel of a row is: with VEC, 8 consecutive channels per j (16-byte
// accesses; C % 8 == 0 and every row 16-byte aligned), else one channel per access, a warp's side
// by side.
template <bool VEC>
__device__ __forceinline__ int channel(int j, int e) {
  const int t = static_cast<int>(blockDim.x), i = static_cast<int>(threadIdx.x);
  return VEC ? (j * t + i) * 8 + e : (j * 8 + e) * t + i;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int j, int C, float (&v)[8]) {
  if (VEC) {
    const int c = channel<true>(j, 0);
    if (c < C) {
      Raw8<T> w;
      w.load(row + c);
      w.unpack(v);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = channel<false>(j, e);
      v[e] = c < C ? to_f32(row[c]) : 0.f;
    }
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int j, int C, const float (&v)[8]) {
  if (VEC) {
    const int c = channel<true>(j, 0);
    if (c < C) {
      Raw8<T> w;
      w.pack(v);
      w.store(row + c);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = channel<false>(j, e);
      if (c < C) row[c] = from_f32<T>(v[e]);
    }
  }
}

// Sums of N values over the CTA, the same in every thread and in a fixed order.  `buf` is one of
// two areas of 32 * N floats used in turn, so one barrier per call is enough.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = static_cast<int>(blockDim.x) >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[i * 32 + w];
}

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
  __shared__ float sums[2][32];
  const int C = a.C;
  const float inv = 1.f / static_cast<float>(C);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float r[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) load8<VEC>(static_cast<const T*>(a.residual) + row * C, j, C, r[j]);
    if (a.block) {
      float b[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) load8<VEC>(static_cast<const T*>(a.block) + row * C, j, C, b[j]);
      if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(b[j][e], b[j][e], s[0]);
        block_sums(s, sums[0]);
        const float bs = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float w[8];
          load8<VEC>(a.post, j, C, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) b[j][e] = b[j][e] * bs * w[e];
        }
      }
      if (a.gate) {
        const T* gr = static_cast<const T*>(a.gate) + row / a.per_gate * C;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float g[8];
          load8<VEC>(gr, j, C, g);
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
      for (int j = 0; j < NV; ++j) store8<VEC>(static_cast<T*>(a.residual_out) + row * C, j, C, r[j]);
    if (a.normed) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(r[j][e], r[j][e], s[0]);
      block_sums(s, sums[1]);
      const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8];
        load8<VEC>(a.pre, j, C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = r[j][e] * rs * w[e];
        store8<VEC>(static_cast<T*>(a.normed) + row * C, j, C, r[j]);
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
  __shared__ float sums[2][3 * 32];
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
      if (part_pre) store8<VEC>(part_pre, j, C, zero);
      if (part_post) store8<VEC>(part_post, j, C, zero);
    }
  }
  float* gate_to = nullptr;  // where the current gate row's sum goes
  for (int64_t row = first; row < last; ++row) {
    const T* const g_row = a.gate ? static_cast<const T*>(a.gate) + row / a.per_gate * C : nullptr;
    if (a.sum_gate && (row == first || row % a.per_gate == 0)) {
      if (SUMS_IN_REGS && gate_to) {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
          store8<VEC>(gate_to, j, C, agate[j]);
#pragma unroll
          for (int e = 0; e < 8; ++e) agate[j][e] = 0.f;
        }
      }
      const int64_t g = row / a.per_gate, begin = g * a.per_gate, end = min(begin + a.per_gate, a.rows);
      if (begin < first) gate_to = a.sum_gate + (cta * 2) * C;
      else if (end > last) gate_to = a.sum_gate + (cta * 2 + 1) * C;
      else gate_to = a.d_gate + g * C;
      if (!SUMS_IN_REGS)
#pragma unroll
        for (int j = 0; j < NV; ++j) store8<VEC>(gate_to, j, C, zero);
    }
    float dr[NV][8], b[NV][8];
    float s[3] = {0.f, 0.f, 0.f};  // r'^2, u r', b^2
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (a.block) {
        load8<VEC>(static_cast<const T*>(a.block) + row * C, j, C, b[j]);
        if (a.post)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[2] = fmaf(b[j][e], b[j][e], s[2]);
      }
      if (a.d_out) {
        load8<VEC>(static_cast<const T*>(a.d_out) + row * C, j, C, dr[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[j][e] = 0.f;
      }
    }
    if (a.d_normed) {
      float r[NV][8], dn[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load8<VEC>(static_cast<const T*>(a.residual_out) + row * C, j, C, r[j]);
        load8<VEC>(static_cast<const T*>(a.d_normed) + row * C, j, C, dn[j]);
        float w[8];
        load8<VEC>(a.pre, j, C, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = fmaf(r[j][e], r[j][e], s[0]);
          s[1] = fmaf(dn[j][e] * w[e], r[j][e], s[1]);
        }
      }
      block_sums(s, sums[0]);
      const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
      const float m = s[1] * inv * rs * rs;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8], add[8];
        load8<VEC>(a.pre, j, C, w);
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
            load8<VEC>(part_pre, j, C, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += add[e];
            store8<VEC>(part_pre, j, C, t);
          }
        }
      }
    } else if (a.post) {
      block_sums(s, sums[0]);
    }
    if (a.d_residual)
#pragma unroll
      for (int j = 0; j < NV; ++j) store8<VEC>(static_cast<T*>(a.d_residual) + row * C, j, C, dr[j]);
    if (a.block) {
      const float bs = a.post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.f;
      float c[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8];
        if (a.post) {
          load8<VEC>(a.post, j, C, w);
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
            load8<VEC>(gate_to, j, C, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += add[e];
            store8<VEC>(gate_to, j, C, t);
          }
        }
        float g[8];
        if (g_row) {
          load8<VEC>(g_row, j, C, g);
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
            load8<VEC>(part_post, j, C, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += add[e];
            store8<VEC>(part_post, j, C, t);
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
        block_sums(c, sums[1]);
        m = c[0] * inv * bs * bs;
      }
      if (a.d_block)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dr[j][e] = bs * (dr[j][e] - b[j][e] * m);
          store8<VEC>(static_cast<T*>(a.d_block) + row * C, j, C, dr[j]);
        }
    }
    if (!a.post) __syncthreads();  // with both reductions, their areas alternate
  }
  if (SUMS_IN_REGS) {
#pragma unroll
    for (int j = 0; j < KV; ++j) {
      if (part_pre) store8<VEC>(part_pre, j, C, apre[j]);
      if (part_post) store8<VEC>(part_post, j, C, apost[j]);
      if (gate_to) store8<VEC>(gate_to, j, C, agate[j]);
    }
  }
}

struct SumArgs {
  const float *sum_pre, *sum_post, *sum_gate;
  float *d_pre, *d_post, *d_gate;
  int64_t rows, per_gate, rows_per_cta;
  int C, ctas;
};

// The partial rows of 32 channels, added in a fixed order.  blockIdx.y: 0 d_pre, 1 d_post, 1 + i the gate
// row that CTA i found begun (and the first to do so).
__global__ void block_norm_sum_kernel(const SumArgs a) {
  __shared__ float part[kSumRows][33];
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
    const int64_t i = y - 1, start = i * a.rows_per_cta, g = start / a.per_gate, begin = g * a.per_gate;
    if (begin == start || begin / a.rows_per_cta + 1 != i) return;
    const int64_t end = min(begin + a.per_gate, a.rows);
    step = 2 * static_cast<int64_t>(a.C);
    from = a.sum_gate + i * step;
    extra = a.sum_gate + (i - 1) * step + a.C;
    n = (end - 1) / a.rows_per_cta - i + 1;
    to = a.d_gate + g * a.C;
  }
  if (!to) return;
  float s = 0.f;
  if (c < a.C) {
    if (extra && threadIdx.y == 0) s = extra[c];
    for (int64_t i = threadIdx.y; i < n; i += kSumRows) s += from[i * step + c];
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

int64_t bwd_ctas(const bconv_block_norm_desc_t* d, int64_t* rows_per_cta) {
  const int64_t most = static_cast<int64_t>(current_sm_count()) * 2;
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

// Calls f.operator()<T, NV, VEC, MAX_THREADS> for a row shape; the bound on the threads keeps the
// registers of the widest rows within what a CTA of that many threads can have.
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
            d->rows,  gate ? d->rows_per_gate : 1, d->width, d->residual_scale, d->eps};
  const bool vec = d->width % 8 == 0 &&
                   all_aligned16({residual, block, gate, post_weight, pre_weight, residual_out, normed});
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
  a.rows = d->rows; a.per_gate = gate ? d->rows_per_gate : 1; a.rows_per_cta = rows_per_cta;
  a.C = d->width; a.alpha = d->residual_scale; a.eps = d->eps;
  const bool vec = d->width % 8 == 0 && all_aligned16({residual_out, block, gate, d_residual_out, d_normed, post_weight,
                                                       pre_weight, d_residual, d_block, d_gate, workspace});
  const Shape sh = shape_for(d->width, 4);
  e = with_dtype(d->dtype,
                 [&](auto t) { return with_shape<decltype(t)>(sh, vec, RunBwd{a, ctas, sh.threads, stream}); });
  if (e != cudaSuccess || !sums) return from_cuda(e);
  SumArgs f{};
  f.sum_pre = a.sum_pre; f.sum_post = a.sum_post; f.sum_gate = a.sum_gate;
  f.d_pre = a.sum_pre ? d_pre_weight : nullptr; f.d_post = d_post_weight; f.d_gate = d_gate;
  f.rows = a.rows; f.per_gate = a.per_gate; f.rows_per_cta = rows_per_cta; f.C = a.C; f.ctas = static_cast<int>(ctas);
  // one grid row more for each CTA boundary that may cut a gate row (1 + i for CTA i)
  const unsigned ys = d_gate ? static_cast<unsigned>(1 + std::max<int64_t>(1, ctas)) : 2u;
  block_norm_sum_kernel<<<dim3(static_cast<unsigned>(ceil_div(a.C, 32)), ys), dim3(32, kSumRows), 0, stream>>>(f);
  return from_cuda(cudaGetLastError());
}

}  // extern "C"
