// The fully-connected layer with 4-bit weights and group scales (bfc_quant_*): entry points,
// the layout of the weights and the choice of kernel.
#include <algorithm>
#include <new>

#include "host_util.cuh"
#include "quant_fc.cuh"

namespace bconv {
namespace {

constexpr uint32_t kQuantMagic = 0x71666334u;
constexpr int kMaxChannels = 1 << 20;
constexpr int64_t kMaxRows = int64_t{1} << 24;

// One 16-byte piece of the laid-out weights per thread (see quant_fc.cuh); codes beyond the
// layer's channels are 0.
__global__ void quant_layout_kernel(const uint8_t* __restrict__ codes, int k, int no, int k_tiles, int64_t pieces,
                                    uint4* __restrict__ out) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= pieces) return;
  const int row_in = static_cast<int>(i % kQuantRows), t = static_cast<int>(i / kQuantRows % 4);
  const int64_t tile = i / (4 * kQuantRows);
  const int kt = static_cast<int>(tile % k_tiles);
  const int64_t row = tile / k_tiles * kQuantRows + row_in;
  const int row_bytes = (k + 1) / 2;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (row < no) {
    const uint8_t* src = codes + row * row_bytes;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k0 = kt * kQuantK + 32 * c + 8 * t;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int kk = k0 + 2 * p;
        if (kk < k) {
          const uint32_t b = src[kk / 2];
          w[c] |= (b & 15u) << (4 * p);
          if (kk + 1 < k) w[c] |= (b >> 4) << (4 * p + 16);
        }
      }
    }
  }
  out[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// [no][groups] -> [groups][no_pad], padding 0
template <typename T>
__global__ void quant_transpose_kernel(const T* __restrict__ src, int no, int no_pad, int groups, T mask,
                                       T* __restrict__ dst) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= static_cast<int64_t>(groups) * no_pad) return;
  const int row = static_cast<int>(i % no_pad);
  const int64_t g = i / no_pad;
  T v = row < no ? src[static_cast<int64_t>(row) * groups + g] : T(0);
  if (sizeof(T) == 1) v = static_cast<T>(static_cast<uint32_t>(v) & static_cast<uint32_t>(mask));
  dst[i] = v;
}

// A device copy of `bytes` at `src` (host or device memory), or `src` itself when it is already on this device.
cudaError_t on_device(const void* src, size_t bytes, int device, void** scratch, const void** p) {
  *scratch = nullptr;
  cudaPointerAttributes at = {};
  const cudaError_t q = cudaPointerGetAttributes(&at, src);
  if (q != cudaSuccess) cudaGetLastError();
  if (q == cudaSuccess && at.type == cudaMemoryTypeDevice && at.device == device) {
    *p = src;
    return cudaSuccess;
  }
  cudaError_t e = cudaMalloc(scratch, bytes);
  if (e == cudaSuccess) e = cudaMemcpy(*scratch, src, bytes, cudaMemcpyDefault);
  *p = *scratch;
  return e;
}

}  // namespace
}  // namespace bconv

struct bfc_quant_handle_s {
  uint32_t magic = 0;
  int device = 0;
  bfc_quant_desc_t desc = {};
  int group = 0, groups = 0, k_tiles = 0, no_pad = 0;
  void* memory = nullptr;  // one allocation: codes, scales, zeros, bias, error word
  uint4* codes = nullptr;
  float* scale = nullptr;
  uint8_t* zero = nullptr;
  float* bias = nullptr;
  uint32_t* err = nullptr;
};

using namespace bconv;

namespace {

bool valid(bfc_quant_handle_t h) { return h && h->magic == kQuantMagic; }

QuantFcArgs args_of(bfc_quant_handle_t h, const void* in, int64_t in_stride, int64_t rows, void* out, int64_t out_stride) {
  QuantFcArgs a{};
  a.codes = h->codes; a.scale = h->scale; a.zero = h->zero; a.bias = h->bias; a.err = h->err;
  a.in = in; a.in_stride = in_stride; a.rows = rows; a.out = out; a.out_stride = out_stride;
  a.k = h->desc.in_channels; a.no = h->desc.out_channels; a.no_pad = h->no_pad;
  a.k_tiles = h->k_tiles; a.group = h->group; a.relu = h->desc.neuron == BCONV_NEURON_RELU;
  return a;
}

cudaError_t fill(bfc_quant_handle_s* h, const uint8_t* codes, const float* scale, const uint8_t* zero,
                 const float* bias) {
  const int k = h->desc.in_channels, no = h->desc.out_channels;
  const int64_t row_tiles = h->no_pad / kQuantRows;
  const int64_t tiles = row_tiles * h->k_tiles, per_group = static_cast<int64_t>(h->groups) * h->no_pad;
  const size_t given = static_cast<size_t>(no) * h->groups;
  void* scratch[3] = {nullptr, nullptr, nullptr};
  const void* src = nullptr;
  const auto blocks = [](int64_t n) { return static_cast<unsigned>(ceil_div(n, 256)); };
  // (every part 256-byte aligned: the kernels copy tiles and groups of channels with bulk copies)
  const auto part = [](int64_t bytes) { return (bytes + 255) / 256 * 256; };
  const int64_t b_codes = part(tiles * kQuantTileBytes), b_scale = part(per_group * 4), b_zero = zero ? part(per_group) : 0,
                b_bias = bias ? part(int64_t{no} * 4) : 0;
  cudaError_t e = cudaMalloc(&h->memory, b_codes + b_scale + b_zero + b_bias + 256);
  if (e != cudaSuccess) return e;
  uint8_t* at = static_cast<uint8_t*>(h->memory);
  h->codes = reinterpret_cast<uint4*>(at);
  h->scale = reinterpret_cast<float*>(at += b_codes);
  h->zero = zero ? (at + b_scale) : nullptr;
  h->bias = bias ? reinterpret_cast<float*>(at + b_scale + b_zero) : nullptr;
  h->err = reinterpret_cast<uint32_t*>(at + b_scale + b_zero + b_bias);
  e = cudaMemsetAsync(h->err, 0, sizeof(uint32_t), nullptr);
  if (e == cudaSuccess) e = on_device(codes, static_cast<size_t>(no) * ((k + 1) / 2), h->device, &scratch[0], &src);
  if (e == cudaSuccess) {
    const int64_t pieces = tiles * 4 * kQuantRows;
    quant_layout_kernel<<<blocks(pieces), 256>>>(static_cast<const uint8_t*>(src), k, no, h->k_tiles, pieces, h->codes);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = on_device(scale, given * sizeof(float), h->device, &scratch[1], &src);
  if (e == cudaSuccess) {
    quant_transpose_kernel<float>
        <<<blocks(per_group), 256>>>(static_cast<const float*>(src), no, h->no_pad, h->groups, 0.f, h->scale);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && zero) {
    e = on_device(zero, given, h->device, &scratch[2], &src);
    if (e == cudaSuccess) {
      quant_transpose_kernel<uint8_t>
          <<<blocks(per_group), 256>>>(static_cast<const uint8_t*>(src), no, h->no_pad, h->groups, uint8_t{15}, h->zero);
      e = cudaGetLastError();
    }
  }
  if (e == cudaSuccess && bias) e = cudaMemcpy(h->bias, bias, no * sizeof(float), cudaMemcpyDefault);
  // the arrays are read during the call only, and any stream may use the handle afterwards
  const cudaError_t done = cudaStreamSynchronize(nullptr);
  for (void* p : scratch)
    if (p) cudaFree(p);
  return e != cudaSuccess ? e : done;
}

}  // namespace

extern "C" {

bconv_status_t bfc_quant_create(const bfc_quant_desc_t* d, const uint8_t* codes, const float* scale,
                                const uint8_t* zero, const float* bias, bfc_quant_handle_t* out) {
  if (!out) return BCONV_ERR_INVALID_ARG;
  *out = nullptr;
  if (!d || !codes || !scale || d->in_channels < 1 || d->out_channels < 1 || d->group_size < 1 ||
      (d->neuron != BCONV_NEURON_NONE && d->neuron != BCONV_NEURON_RELU) || !valid_dtype(d->in_dtype) ||
      !valid_dtype(d->out_dtype) || !aligned_elem(scale, BCONV_DTYPE_F32) || !aligned_elem(bias, BCONV_DTYPE_F32))
    return BCONV_ERR_INVALID_ARG;
  if (d->in_channels > kMaxChannels || d->out_channels > kMaxChannels) return BCONV_ERR_UNSUPPORTED;
  const bool whole = d->group_size >= d->in_channels;
  if (!whole && d->group_size != 32 && d->group_size != 64 && d->group_size % kQuantK != 0)
    return BCONV_ERR_UNSUPPORTED;
  int device = 0;
  const cudaError_t found = cudaGetDevice(&device);
  if (found != cudaSuccess) {
    cudaGetLastError();
    return from_cuda(found);
  }
  bfc_quant_handle_s* h = new (std::nothrow) bfc_quant_handle_s();
  if (!h) return BCONV_ERR_OOM;
  h->magic = kQuantMagic;
  h->device = device;
  h->desc = *d;
  h->k_tiles = (d->in_channels + kQuantK - 1) / kQuantK;
  h->group = whole ? h->k_tiles * kQuantK : d->group_size;
  h->groups = (d->in_channels + h->group - 1) / h->group;
  h->no_pad = round_up(d->out_channels, kQuantRows);
  const cudaError_t e = fill(h, codes, scale, zero, bias);
  if (e != cudaSuccess) {
    cudaGetLastError();
    h->magic = 0;
    cudaFree(h->memory);
    delete h;
    return from_cuda(e);
  }
  *out = h;
  return BCONV_OK;
}

int64_t bfc_quant_workspace_bytes(bfc_quant_handle_t h, const void* in, int64_t in_stride, int64_t rows) {
  if (!valid(h) || rows < 0 || rows > kMaxRows || in_stride < h->desc.in_channels) return -1;
  if (rows == 0 || quant_fc_tma_reads(in, in_stride, h->desc.in_channels, h->desc.in_dtype) ||
      quant_fc_rows_serves(args_of(h, in, in_stride, rows, nullptr, 0), h->desc.in_dtype))
    return 0;
  return quant_fc_tc_workspace(rows, h->desc.in_channels, h->desc.in_dtype);
}

bconv_status_t bfc_quant_forward(bfc_quant_handle_t h, const void* in, int64_t in_stride, int64_t rows, void* out,
                                 int64_t out_stride, void* workspace, struct CUstream_st* stream) {
  if (!valid(h) || rows < 0 || rows > kMaxRows || in_stride < h->desc.in_channels ||
      out_stride < h->desc.out_channels || !aligned_elem(in, h->desc.in_dtype) ||
      !aligned_elem(out, h->desc.out_dtype) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BCONV_ERR_INVALID_ARG;
  if (rows == 0) return BCONV_OK;
  if (!in || !out || (!workspace && bfc_quant_workspace_bytes(h, in, in_stride, rows) > 0)) return BCONV_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return BCONV_ERR_CUDA;
  const QuantFcArgs a = args_of(h, in, in_stride, rows, out, out_stride);
  if (quant_fc_rows_serves(a, h->desc.in_dtype))
    return from_cuda(launch_quant_fc_rows(a, h->desc.in_dtype, h->desc.out_dtype, stream));
  return from_cuda(launch_quant_fc_tc(a, h->desc.in_dtype, h->desc.out_dtype, workspace, stream));
}

int32_t bfc_quant_input_feature_channels(bfc_quant_handle_t h) { return valid(h) ? h->desc.in_channels : -1; }
int32_t bfc_quant_output_feature_channels(bfc_quant_handle_t h) { return valid(h) ? h->desc.out_channels : -1; }

bconv_status_t bfc_quant_sync_status(bfc_quant_handle_t h, struct CUstream_st* stream) {
  if (!valid(h)) return BCONV_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return BCONV_ERR_CUDA;
  uint32_t err = 0;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpy(&err, h->err, sizeof(err), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && err) e = cudaMemset(h->err, 0, sizeof(err));
  if (e != cudaSuccess) return from_cuda(e);
  return err & kErrTimeout ? BCONV_ERR_TIMEOUT : err ? BCONV_ERR_CUDA : BCONV_OK;
}

bconv_status_t bfc_quant_destroy(bfc_quant_handle_t h) {
  if (!h) return BCONV_OK;
  if (!valid(h)) return BCONV_ERR_INVALID_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return BCONV_ERR_CUDA;
  const cudaError_t e = cudaDeviceSynchronize();
  h->magic = 0;
  cudaFree(h->memory);
  delete h;
  return from_cuda(e);
}

}  // extern "C"
