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

// Codes less zeros, exactly: the four pairs of a word of codes.  A pair lies in the low bits of the halves of a
// register and is or-ed into 1024.0 (fp16) or 128.0 (bf16), whose last significant bits are worth 1; `zero`, that
// constant plus the zero, twice, is taken off.  One three-operand logic instruction takes the bits out and puts them in
// (two constants at once are more than an instruction can name, so one is given in a register).  fp16 has room for
// the pair above too: 1024 + 16 code, which one multiply-add makes 64 + code - (64 + zero); that saves two of the
// three shifts.  (bf16 holds 7 bits behind the point, too few for two.)
__device__ __forceinline__ uint32_t take(uint32_t w, uint32_t mask, uint32_t bias) {
  uint32_t a;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(a) : "r"(w), "r"(mask), "r"(bias));  // (w & mask) | bias
  return a;
}
template <bool HALF>
__device__ __forceinline__ void decode(uint32_t w, uint32_t zero, uint32_t (&p)[4]) {
  if (HALF) {
    const uint32_t high = take(zero << 4, 0x00f000f0u, 0xd400d400u), sixteenth = 0x2c002c00u;  // -(64 + zero), 1 / 16
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = i ? w >> 8 : w;
      const uint32_t a = take(v, 0x000f000fu, 0x64006400u), b = take(v, 0x00f000f0u, 0x64006400u);
      const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&zero));
      const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&sixteenth),
                                *reinterpret_cast<const __half2*>(&high));
      p[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
      p[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = take(w >> (4 * i), 0x000f000fu, 0x43004300u);
      const __nv_bfloat162 r =
          __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&zero));
      p[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
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
