// The 4-bit fully-connected layer on the SIMT units: one thread per output channel and row.
//
//     out[r][c] = act( sum_groups scale[c][g] * sum_{f in g} in[r][f] * (code[c][f] - zero[c][g]) + bias[c] )
//
// A CTA is one row and one tile of 128 output channels; it stages 128 inputs at a time in shared
// memory, where every thread reads the same one, and each thread decodes its own channel's
// 64 bytes of the weight tile.
#include "quant_fc.cuh"

namespace bconv {
namespace {

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kQuantRows) quant_fc_simt_kernel(const QuantFcArgs a) {
  __shared__ float x[kQuantK];
  const int64_t r = blockIdx.y;
  const int c = blockIdx.x * kQuantRows + threadIdx.x;
  const TIn* in = static_cast<const TIn*>(a.in) + r * a.in_stride;
  const uint4* tile = a.codes + static_cast<int64_t>(blockIdx.x) * a.k_tiles * (kQuantTileBytes / 16);
  float acc = 0.f;
  for (int kt = 0; kt < a.k_tiles; ++kt, tile += kQuantTileBytes / 16) {
    __syncthreads();
    const int f = kt * kQuantK + threadIdx.x;
    x[threadIdx.x] = f < a.k ? to_f32(in[f]) : 0.f;
    __syncthreads();
    uint32_t w[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint4 v = tile[t * kQuantRows + threadIdx.x];
      w[t][0] = v.x; w[t][1] = v.y; w[t][2] = v.z; w[t][3] = v.w;
    }
#pragma unroll
    for (int c4 = 0; c4 < 4; ++c4) {  // 32 channels: within one group
      const int k0 = kt * kQuantK + 32 * c4;
      if (k0 >= a.k) break;
      const int64_t g = static_cast<int64_t>(k0 / a.group) * a.no_pad + c;
      const int z = a.zero ? a.zero[g] : 8;
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t v = w[t][c4] >> (4 * p);
          s = fmaf(x[32 * c4 + 8 * t + 2 * p], static_cast<float>(static_cast<int>(v & 15u) - z), s);
          s = fmaf(x[32 * c4 + 8 * t + 2 * p + 1], static_cast<float>(static_cast<int>((v >> 16) & 15u) - z), s);
        }
      acc = fmaf(a.scale[g], s, acc);
    }
  }
  if (c < a.no) {
    if (a.bias) acc += a.bias[c];
    if (a.relu) acc = acc < 0.f ? 0.f : acc;
    static_cast<TOut*>(a.out)[r * a.out_stride + c] = from_f32<TOut>(acc);
  }
}

}  // namespace

cudaError_t launch_quant_fc_simt(const QuantFcArgs& a, int in_dtype, int out_dtype, cudaStream_t s) {
  return with_dtype(in_dtype, [&](auto ti) {
    return with_dtype(out_dtype, [&](auto to) {
      // (grid rows are limited to 65535)
      constexpr int64_t kMost = 65535;
      for (int64_t r = 0; r < a.rows; r += kMost) {
        QuantFcArgs b = a;
        b.rows = a.rows - r < kMost ? a.rows - r : kMost;
        b.in = static_cast<const decltype(ti)*>(a.in) + r * a.in_stride;
        b.out = static_cast<decltype(to)*>(a.out) + r * a.out_stride;
        quant_fc_simt_kernel<decltype(ti), decltype(to)>
            <<<dim3(static_cast<unsigned>(a.no_pad / kQuantRows), static_cast<unsigned>(b.rows)), kQuantRows, 0, s>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
      }
      return cudaSuccess;
    });
  });
}

}  // namespace bconv
