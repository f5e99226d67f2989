// The 4-bit fully-connected layer for few rows (at most 16): every code is read once, straight into
// registers.
//
// A warp owns 16 output channels and a share of the input channels; its codes pass through a ring of
// registers (kDepth tiles of 128 input channels ahead), become the A operand of m16n8k16 MMAs (code -
// zero: whole numbers, exact in bf16 and fp16) and meet the rows, which lie in shared memory as the B
// operand: tokens are the columns, 8 to an MMA.  As in the tensor-core kernel a group's sum is
// scaled and added in fp32, and fp32 inputs come as three bf16 parts.  The layout of the codes makes
// 16 bytes of a row exactly what the MMA's lanes want: word c of lane t holds channels 32 c + 8 t .. + 7, two
// MMAs' worth, and the lane's B operands for them are 16 consecutive bytes of the row.
//
// Warps of a CTA share a channel tile's input channels (ksplit of them) where there are too few
// tiles to fill the SMs, and add up their sums through shared memory in a fixed order.
//
// The rows lie in shared memory as a whole, 100 KB at most: 12 rows of 4096 channels in 16 bits, 4 in fp32; what does
// not fit takes the tensor-core kernel, one step of which costs more (16 x 4096 -> 16384 bf16 20.9 us, 12 rows 17.6).
//
// HBM is not what bounds it: 1 x 4096 x 65536 bf16 38 us (3.7 TB/s), fp16 35.7 (3.9 TB/s), 1 x 4000 x 65537 fp16 with
// zeros for groups of 64 45.6.  Neither are the issue slots (54 % bf16, 49 % fp16 with groups of 64) nor the integer
// units that take the codes out of their words (53 %, 41 %) full: the 16 warps an SM wait for one another's results, for
// codes, and, with small groups, for scales and zeros, of which the ring holds two tiles instead of four.  The
// 5th-generation tensor cores would have nothing to gain here: their operands pass through TMEM, one more
// step for every code (with that kernel 68, 66 and 76 us, its MMAs idle most of the time).
#include <algorithm>
#include <type_traits>

#include "host_util.cuh"
#include "quant_fc.cuh"

namespace bconv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSmem = 100 * 1024;  // of the rows: two CTAs an SM, but for the largest calls of 9 to 16 rows

// CTAs that an SM's 228 KB hold: of `smem` bytes for the rows each, the sums of nt tiles of 8 tokens, and the 1 KB that
// the hardware keeps.
constexpr int sums_bytes(int nt) { return 2 * kWarps * nt * 4 * 32 * 4; }
constexpr int ctas_per_sm(int smem, int nt) {
  return std::max(1, std::min(2, 228 * 1024 / (smem + sums_bytes(nt) + 1024)));
}
static_assert(ctas_per_sm(kMaxSmem, 1) == 2 && ctas_per_sm(97 * 1024, 2) == 2 && ctas_per_sm(98 * 1024, 2) == 1, "");

struct RowsArgs {
  QuantFcArgs q;
  int ksplit;      // warps sharing a channel tile
  int k_each;      // tiles of 128 input channels of a warp
  int tiles;       // channel tiles of 16
  int pitch;       // bytes between the rows in shared memory
};

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (HALF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile of 128 input channels of this lane's two channels.
template <int UNITS, bool ZERO>
struct Item {
  uint4 w[2];
  float s[2][UNITS];
  uint32_t z[2][ZERO ? UNITS : 1];
};

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// T: element type of the rows; PARTS: 1, or 3 bf16 parts of fp32; NT: tiles of 8 tokens; UNITS: groups per 128
// input channels; ZERO: whether the layer has zeros (else they are 8).
template <typename T, int PARTS, int NT, int UNITS, bool ZERO>
__global__ void __launch_bounds__(kThreads, 2) quant_fc_rows_kernel(const RowsArgs a, int out_dtype) {
  constexpr bool HALF = std::is_same<T, __half>::value;
  constexpr uint32_t kBias = HALF ? 0x6400u : 0x4300u;  // 1024.0 or 128.0: or-ing a 4-bit number in adds it
  constexpr int kDepth = UNITS == 1 ? 4 : 2;
  extern __shared__ __align__(16) uint8_t smem[];  // [part][row][pitch], 256 bytes of zeros
  __shared__ float sums[2][kWarps][NT * 4][32];  // sums_bytes(NT); used in turn, so that one barrier a tile is enough
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rows = static_cast<int>(a.q.rows);
  const int share = warp % a.ksplit, team = warp / a.ksplit, teams = kWarps / a.ksplit;
  const int kt0 = min(share * a.k_each, a.q.k_tiles), nk = min(kt0 + a.k_each, a.q.k_tiles) - kt0;

  // items: tile after tile, nk steps each.  The addresses of the next one to load move on by additions.
  const int stride = gridDim.x * teams, first = blockIdx.x * teams + team;
  Item<UNITS, ZERO> ring[kDepth];
  int l_tile = first, l_k = 0, l_group = 0, l_left = 0;  // l_left: steps until the next group (one unit)
  const uint4* l_codes = nullptr;
  const float* l_scale = nullptr;
  const uint8_t* l_zero = nullptr;
  const int last_group = (a.q.k + a.q.group - 1) / a.q.group - 1;
  const int steps_per_group = a.q.group / kQuantK;  // (one unit)
  auto start_tile = [&]() {
    const int row = l_tile * 16 + g;
    l_codes = a.q.codes + (static_cast<int64_t>(row / kQuantRows) * a.q.k_tiles + kt0) * (kQuantTileBytes / 16) +
              t * kQuantRows + row % kQuantRows;
    l_group = UNITS == 1 ? kt0 / steps_per_group : kt0 * UNITS;
    l_left = UNITS == 1 ? steps_per_group - (kt0 - l_group * steps_per_group) : 0;
    const int64_t terms = static_cast<int64_t>(min(l_group, last_group)) * a.q.no_pad + row;
    l_scale = a.q.scale + terms;
    if (ZERO) l_zero = a.q.zero + terms;
  };
  auto load = [&](Item<UNITS, ZERO>& it) {
    if (l_tile >= a.tiles) return;
    it.w[0] = __ldcs(l_codes);
    it.w[1] = __ldcs(l_codes + 8);
    l_codes += kQuantTileBytes / 16;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      it.s[0][u] = __ldg(l_scale);
      it.s[1][u] = __ldg(l_scale + 8);
      if (ZERO) {
        it.z[0][u] = __ldg(l_zero);
        it.z[1][u] = __ldg(l_zero + 8);
      }
      // (behind the last group the inputs are 0)
      if (UNITS > 1 || --l_left == 0) {
        if (l_group++ < last_group) {
          l_scale += a.q.no_pad;
          if (ZERO) l_zero += a.q.no_pad;
        }
        l_left = steps_per_group;
      }
    }
    if (++l_k == nk) {
      l_k = 0;
      l_tile += stride;
      start_tile();
    }
  };
  if (nk == 0) l_tile = a.tiles;
  start_tile();
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ring[i]);

  // the rows into shared memory, 8 channels at a time, channels behind the last as 0
  const int plane = rows * a.pitch;
  if (threadIdx.x < 16) *reinterpret_cast<uint4*>(smem + PARTS * plane + threadIdx.x * 16) = make_uint4(0u, 0u, 0u, 0u);
  wait_prior_grid();
  {
    const int octets = a.q.k_tiles * (kQuantK / 8), total = rows * octets;
    const bool vec = (reinterpret_cast<uintptr_t>(a.q.in) & 15u) == 0 && a.q.in_stride % 8 == 0;
    constexpr int kBatch = 4;  // loads in flight together
    for (int base = threadIdx.x; base < total; base += kBatch * kThreads) {
      Raw8<T> x[kBatch];
      int at[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = base + b * kThreads, r = i / octets, c = (i - r * octets) * 8;
        at[b] = r * a.pitch + c * 2;
        const T* in = static_cast<const T*>(a.q.in) + r * a.q.in_stride + c;
        if (i < total && vec && c + 8 <= a.q.k) {
          x[b].load(in);
        } else {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = i < total && c + e < a.q.k ? to_f32(in[e]) : 0.f;
          x[b].pack(v);  // (back to the same bits)
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (base + b * kThreads >= total) break;
        if constexpr (PARTS == 3) {
          float v[8];
          uint32_t p[3][4];
          x[b].unpack(v);
#pragma unroll
          for (int e = 0; e < 4; ++e) split3_bf16x2(v[2 * e], v[2 * e + 1], p[0][e], p[1][e], p[2][e]);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4*>(smem + q * plane + at[b]) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
        } else {
          *reinterpret_cast<uint4*>(smem + at[b]) = x[b].w;
        }
      }
    }
  }
  __syncthreads();
  allow_next_grid();

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  const int turns = (a.tiles - static_cast<int>(blockIdx.x) * teams + stride - 1) / stride;  // of the CTA's first team
  int tile = first, k = 0;
  // this lane's B operands: row n * 8 + g, or zeros (256 bytes behind the rows) where there is no such row
  uint32_t x_start[NT], x_at[NT], x_step[NT], x_plane[NT];
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const bool real = n * 8 + g < rows;
    x_start[n] = x_at[n] = base + (real ? (n * 8 + g) * a.pitch + (kt0 * kQuantK + 8 * t) * 2 : PARTS * plane + 16 * t);
    x_step[n] = real ? kQuantK * 2 : 0;
    x_plane[n] = real ? plane : 0;
  }

  int turn = 0;
  auto finish = [&]() {  // the tile's sums are complete (nothing in warps without input channels)
    const bool real = tile < a.tiles;
    if (a.ksplit > 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[turn][warp][n * 4 + i][lane] = acc[n][i];
      __syncthreads();
    }
    if (share == 0 && real) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[n][i];
          for (int p = 1; p < a.ksplit; ++p) v += sums[turn][warp + p][n * 4 + i][lane];
          const int c = tile * 16 + g + (i >= 2 ? 8 : 0), row = n * 8 + 2 * t + (i & 1);
          if (c < a.q.no && row < rows) {
            if (a.q.bias) v += __ldg(a.q.bias + c);
            if (a.q.relu) v = v < 0.f ? 0.f : v;
            const int64_t at = row * a.q.out_stride + c;
            if (out_dtype == BCONV_DTYPE_F32) static_cast<float*>(a.q.out)[at] = v;
            else if (out_dtype == BCONV_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.q.out)[at] = __float2bfloat16_rn(v);
            else static_cast<__half*>(a.q.out)[at] = __float2half_rn(v);
          }
        }
    }
    turn ^= 1;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    tile += stride;
  };

  auto step = [&](const Item<UNITS, ZERO>& it) {
    const uint32_t w[2][4] = {{it.w[0].x, it.w[0].y, it.w[0].z, it.w[0].w}, {it.w[1].x, it.w[1].y, it.w[1].z, it.w[1].w}};
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint32_t zz[2] = {ZERO ? (kBias | it.z[0][u]) * 0x10001u : (kBias | 8u) * 0x10001u,
                              ZERO ? (kBias | it.z[1][u]) * 0x10001u : (kBias | 8u) * 0x10001u};
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[n][i] = 0.f;
#pragma unroll
      for (int c = u * (4 / UNITS); c < (u + 1) * (4 / UNITS); ++c) {
        uint32_t p[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) decode<HALF>(w[r][c], zz[r], p[r]);
        const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]}, a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 b = lds128(x_at[n] + part * x_plane[n] + c * 64);
            mma16816<HALF>(d[n], a0, b.x, b.y);
            mma16816<HALF>(d[n], a1, b.z, b.w);
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(it.s[i >> 1][u], d[n][i], acc[n][i]);
    }
  };

  if (nk == 0) {
    for (int i = 0; i < turns; ++i) finish();
    return;
  }
  // (every warp of a CTA finishes `turns` tiles, real or not, so that the barriers meet; tiles behind the last
  // repeat old codes, and nothing of them is written)
  int done = 0;
  while (done < turns) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (done < turns) {
        step(ring[i]);
        load(ring[i]);
#pragma unroll
        for (int n = 0; n < NT; ++n) x_at[n] += x_step[n];
        if (++k == nk) {
          k = 0;
#pragma unroll
          for (int n = 0; n < NT; ++n) x_at[n] = x_start[n];
          finish();
          ++done;
        }
      }
    }
  }
}

template <typename T, int PARTS, int NT, int UNITS, bool ZERO>
cudaError_t launch(const RowsArgs& a, int out_dtype, int ctas, int smem, cudaStream_t s) {
  auto kern = quant_fc_rows_kernel<T, PARTS, NT, UNITS, ZERO>;
  const cudaError_t set = allow_smem<quant_fc_rows_kernel<T, PARTS, NT, UNITS, ZERO>>(kMaxSmem);
  if (set != cudaSuccess) return set;
  const cudaError_t e = launch_overlapped(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, s, a, out_dtype);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Bytes between rows in shared memory: 64 off a multiple of 128, so that the 8 lanes of an access (two rows of 64
// bytes) meet different banks.
int pitch_for(const QuantFcArgs& q) { return round_up(q.k_tiles * kQuantK * 2, 128) + 64; }
int smem_for(const QuantFcArgs& q, int in_dtype) {
  return pitch_for(q) * static_cast<int>(q.rows) * (in_dtype == BCONV_DTYPE_F32 ? 3 : 1) + 256;
}

}  // namespace

bool quant_fc_rows_serves(const QuantFcArgs& q, int in_dtype) {
  return q.rows <= 16 && static_cast<int64_t>(pitch_for(q)) * q.rows * 3 < (1 << 28) && smem_for(q, in_dtype) <= kMaxSmem;
}

cudaError_t launch_quant_fc_rows(const QuantFcArgs& q, int in_dtype, int out_dtype, cudaStream_t s) {
  RowsArgs a{};
  a.q = q;
  a.pitch = pitch_for(q);
  a.tiles = (q.no + 15) / 16;
  const int smem = smem_for(q, in_dtype);
  const int units = q.group >= kQuantK ? 1 : kQuantK / q.group;
  // warps per tile: the split that finishes first with the CTAs that are resident, the end of a shared tile costing
  // about one step for every 8 tokens
  const int nt = q.rows <= 8 ? 1 : 2, slots = ctas_per_sm(smem, nt) * current_sm_count();
  double best = 1e300;
  int ctas = 1;
  for (int ks = 1; ks <= kWarps; ks *= 2) {
    const int teams = kWarps / ks, work = (a.tiles + teams - 1) / teams, each = (q.k_tiles + ks - 1) / ks;
    const double cost = static_cast<double>((work + slots - 1) / slots) * (each + (ks > 1 ? nt : 0.5));
    if (cost < best * 0.97) {
      best = cost;
      a.ksplit = ks;
      a.k_each = each;
      ctas = std::min(work, slots);
    }
  }
  const auto with_units = [&](auto t, auto parts, auto nt) {
    using T = decltype(t);
    constexpr int kParts = decltype(parts)::value, kNt = decltype(nt)::value;
    const auto with_zero = [&](auto has) {
      constexpr bool kZero = decltype(has)::value;
      switch (units) {
        case 1: return launch<T, kParts, kNt, 1, kZero>(a, out_dtype, ctas, smem, s);
        case 2: return launch<T, kParts, kNt, 2, kZero>(a, out_dtype, ctas, smem, s);
        default: return launch<T, kParts, kNt, 4, kZero>(a, out_dtype, ctas, smem, s);
      }
    };
    return q.zero ? with_zero(std::true_type{}) : with_zero(std::false_type{});
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Three = std::integral_constant<int, 3>;
  const bool one = q.rows <= 8;
  if (in_dtype == BCONV_DTYPE_F32) return one ? with_units(float{}, Three{}, One{}) : with_units(float{}, Three{}, Two{});
  if (in_dtype == BCONV_DTYPE_BF16)
    return one ? with_units(__nv_bfloat16{}, One{}, One{}) : with_units(__nv_bfloat16{}, One{}, Two{});
  return one ? with_units(__half{}, One{}, One{}) : with_units(__half{}, One{}, Two{});
}

}  // namespace bconv
