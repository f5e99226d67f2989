// The fully-connected layer with 4-bit weights: its handle, and the layout of its weights that
// the kernels share; internal.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "dtype.cuh"

namespace bconv {

// Weights lie in tiles of kQuantRows output channels x kQuantK input channels (8 KB), [row
// tile][k tile].  A tile is [t = 0..3][row][16 bytes]: word c = 0..3 of piece t of a row holds
// input channels 32 c + 8 t .. + 7, and within a word channel 2 p is nibble p and channel 2 p + 1
// nibble p + 4, so that (word >> 4 p) & 0x000f000f is a pair of neighbours in the halves of a
// 32-bit register.  Word c of the pieces of a row is 32 consecutive channels, the smallest
// group; lanes that take one piece each of consecutive rows read consecutive 16-byte pieces.
constexpr int kQuantRows = 128;
constexpr int kQuantK = 128;
constexpr int kQuantTileBytes = kQuantRows * kQuantK / 2;

struct QuantFcArgs {
  const uint4* codes;     // [row tiles][k tiles] tiles
  const float* scale;     // [groups][no_pad]
  const uint8_t* zero;    // [groups][no_pad] or NULL (8)
  const float* bias;      // [no] or NULL
  const void* in;
  void* out;
  uint32_t* err;
  int64_t in_stride, out_stride, rows;
  int k, no, no_pad;      // no_pad: a multiple of kQuantRows
  int k_tiles, group;     // group: input channels per scale
  int relu;
};

// Whether the tensor-core kernel reads these rows as they are (else they are staged in the workspace,
// of quant_fc_tc_workspace bytes).
bool quant_fc_tma_reads(const void* in, int64_t in_stride, int k, int in_dtype);
int64_t quant_fc_tc_workspace(int64_t rows, int k, int in_dtype);
cudaError_t launch_quant_fc_tc(const QuantFcArgs& a, int in_dtype, int out_dtype, void* workspace, cudaStream_t s);

}  // namespace bconv
