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

// Codes less zeros: two 4-bit numbers of w, in the low bits of its halves, or-ed into 1024.0 (fp16) or 128.0
// (bf16), whose last significant bits are worth 1, less `zero`, that constant plus the zero, twice.  Exact.  One
// three-operand logic instruction takes the bits out and puts them in (two constants at once are more than
// an instruction can name, so one is given in a register).
template <bool HALF>
__device__ __forceinline__ uint32_t decode(uint32_t w, uint32_t zero) {
  uint32_t a;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a) : "r"(w), "r"(0x000f000fu), "r"(HALF ? 0x64006400u : 0x43004300u));
  if (HALF) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&zero));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&zero));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// At most 16 rows that fit in shared memory.
bool quant_fc_rows_serves(const QuantFcArgs& q, int in_dtype);
cudaError_t launch_quant_fc_rows(const QuantFcArgs& q, int in_dtype, int out_dtype, cudaStream_t s);
// Whether the tensor-core kernel reads these rows as they are (else they are staged in the workspace,
// of quant_fc_tc_workspace bytes).
bool quant_fc_tma_reads(const void* in, int64_t in_stride, int k, int in_dtype);
int64_t quant_fc_tc_workspace(int64_t rows, int k, int in_dtype);
cudaError_t launch_quant_fc_tc(const QuantFcArgs& a, int in_dtype, int out_dtype, void* workspace, cudaStream_t s);

}  // namespace bconv
