// The 4-bit fully-connected layer on the 5th-generation tensor cores.
//
//     out[r][c] = act( sum_g scale[c][g] * ( sum_{f in g} (code[c][f] - zero[c][g]) * in[r][f] ) + bias[c] )
//
// The roles of the operands are swapped: the 128 output channels of a tile are the M rows of the
// MMA and the tokens its N columns, so few tokens waste no tensor work, and a TMEM lane belongs to one
// channel: a group's scale is one register per thread.  code - zero is a whole number of at most 15
// and exact in bf16 and fp16, so the tensor cores sum exact products of the input (kind::f16 with
// fp32 accumulators) and every group's sum is scaled and added in fp32 registers; no weight is
// ever rounded.  fp32 inputs come as three bf16 parts whose sum they are (see stage_kernel), each
// multiplied by the same codes: one after the other into the same sums, or, for up to 32 rows, as three times as many
// tokens (9 rows of 25088 channels: a third of the MMAs).
//
// The codes become operands in TMEM, not in shared memory: eight warps read a tile's packed codes (8
// KB per 128 x 128, one bulk copy) and write them with tcgen05.st as the MMA's A operand, one
// channel per lane.  Through shared memory they would cost 4 times the packed bytes in and again out of
// it per tile, more than its 128 bytes a cycle for up to about 100 tokens.
//
// Roles (20 warps): warp 0 loads the tokens (TMA boxes of 64 input channels x N tokens) and the scales,
// warp 1 issues the MMAs, warp 2 loads the codes, warps 4-7 and 8-11 decode every second tile,
// warps 12-15 and 16-19 take the groups' sums out of TMEM: up to 96 tokens those of every second group
// each, with two accumulators each; above, half of the tokens of every group each, with two accumulators
// in turn, so that one sum is taken out while the next one is formed.  The one thread that issues the MMAs is
// on the critical path: up to 64 tokens a tile takes it about 600 of the 800 cycles that the tile takes in all.  So
// the MMAs are few and large (160 x 4096 x 16384 bf16: 28.9 us with MMAs of 160 tokens, 30.9 with two of
// 80), and the barriers few: one per tile for everything that the MMAs read (tokens, scales, codes) and
// one for its release, and two per accumulator.
// A CTA walks over its tiles without a pause: tokens and codes of the next one are on their way and decoded
// while the sums of the last are written (a CTA per tile spent 8 us a tile outside its loop over
// the input channels: 44 of 140 us for 2000 x 4096 x 8192).  Where there are few tiles, a cluster of CTAs
// shares a tile's input channels and adds up its parts over distributed shared memory in rank order.
//
// No unit is full.  For many tokens the tensor cores (4 N cycles per 128 input channels) are busy most (2000 x 4096 ->
// 8192 bf16: 55 %, issue slots 52 %; 160 x 4096 -> 16384: 41 % and 47 %), for few the chain of decoding a tile, its MMAs
// and taking out their sums is (9 x 25088 -> 4096 fp32: tensor cores 10 %, issue slots 40 %, HBM 19 %); warps wait most
// for loads, those from TMEM among them.  Groups of 32 and 64 have two and four times as many sums to take out, fp32 rows
// above 32 three times the MMAs on at most 64 tokens (160 x 4096 -> 16384 fp32 81 us, 2000 x 4096 -> 8192 374).
// Every wait gives up after one second, sets the error word and makes all roles stop.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <stddef.h>

#include <algorithm>
#include <type_traits>

#include "elect.cuh"
#include "f32x2.cuh"
#include "host_util.cuh"
#include "quant_fc.cuh"
#include "tc_device.cuh"

namespace bconv {
namespace {

using namespace tcdev;

constexpr int kThreads = 640;
constexpr int kWStages = 6;          // tiles of codes in flight
constexpr int kMaxStages = 8;        // tiles of tokens in flight
constexpr int kScaleSlack = 4;       // the scales of a tile are used up to so many tiles after its tokens
constexpr int kMaxCols = 96;         // tokens whose sums a warp takes out; two warpgroups may share an MMA's
constexpr int kSlots = 4;            // accumulators of up to kMaxCols tokens, or two of twice as many
constexpr int kACols = kQuantK / 2;  // TMEM columns of a decoded tile
constexpr int kTmemCols = 512;
static_assert(kSlots * kMaxCols + 2 * kACols <= kTmemCols, "TMEM: a decoded tile of each decoding warpgroup at least");
constexpr int kMaxSplit = 8;
constexpr int kSmemBytes = 226 * 1024;

struct __align__(16) Bars {
  uint64_t ready[kMaxStages];  // a tile's tokens and scales (bytes) and its four decoding warps
  uint64_t done[kMaxStages];   // its MMAs
  uint64_t full_w[kWStages], empty_w[kWStages];
  uint64_t full_d[kSlots], empty_d[kSlots];
  uint64_t last;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

// shared memory: [tokens][exchange][codes, zeros][scales] in whole KB, the barriers behind them
constexpr int kRingBytes = (kSmemBytes - static_cast<int>(sizeof(Bars))) / 1024 * 1024;

struct TcQuantArgs {
  QuantFcArgs q;
  int cols;        // tokens of an MMA: a multiple of 16 up to kMaxCols, or of 32 up to twice that
  int slot_cols;   // TMEM columns between the accumulators
  int a_stages;    // decoded tiles in TMEM (even: the decoding warpgroups take turns)
  int parts;       // bf16 parts of the input (3 for fp32), multiplied one after the other
  int fold;        // or 3 parts as rows of their own, whose sums are added up at the end
  int part_rows;   // rows between the parts in the tensor map
  int stages;      // tiles of tokens in flight
  int tiles;       // of 128 channels x cols tokens
  int exchange;    // bytes for the sums of the second stream (one half of tokens, CTAs of several tiles)
  int units;       // groups per 128 input channels (1 for groups of 128 and more)
  int splits;      // CTAs of a cluster sharing a tile
  int out_dtype;
  int staged;      // the input is written by the kernel before this one
};

// Codes of a tile and the zeros of its groups.
__host__ __device__ constexpr int w_stage_bytes(int units, bool zero) {
  return kQuantTileBytes + (zero ? units * kQuantRows : 0);
}

// D += A * B^T, A (128 x 16, 16-bit) in TMEM, B (N x 16) in shared memory, fp32 accumulator.  The
// descriptor of B (128-byte rows and swizzle) is given by its low word; see smem_desc_sw128.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ts_add(uint32_t d, uint32_t a, uint32_t b_desc_low, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, 1, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_desc_low), "r"(idesc), "n"(kDescHigh)
      : "memory");
}
// The same, or D = A * B^T, as known only at run time.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_desc_low, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_desc_low), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "n"(kDescHigh)
      : "memory");
}

// 32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void st_32x32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// 16 columns of this warp's 32 TMEM lanes; the values may be used after ld_wait of the same registers.
__device__ __forceinline__ void ld_16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void ld_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Barriers by their shared-memory address: what a single thread does between two MMAs is on the
// critical path, instruction by instruction.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The rest of a wait that did not succeed at once.  The clock is read only after many tries: reading it
// costs more than a usual wait.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Bars* B, uint32_t* err) {
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
      if (try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile uint32_t*>(&B->abort_flag)) return false;
    const uint64_t t = globaltimer();
    if (t0 == 0) t0 = t;
    if (t - t0 > kTimeoutNs) {
      atomicOr(err, kErrTimeout);
      atomicExch(&B->abort_flag, 1u);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Bars* B, uint32_t* err) {
  return try_wait(bar, parity) || wait_slow(bar, parity, B, err);
}
// The same for a whole warp, all lanes together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, Bars* B, uint32_t* err) {
  if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_slow(bar, parity, B, err));
}

// After giving up: wait (for a second at most) until the last `issued` copies of a ring have landed.
__device__ __forceinline__ void drain(uint64_t* full, int stages, int issued) {
  const uint64_t t0 = globaltimer();
  for (int i = max(0, issued - stages); i < issued; ++i)
    while (!mbar_try_suspend(&full[i % stages], static_cast<uint32_t>(i / stages) & 1u, 20000u))
      if (globaltimer() - t0 > kTimeoutNs) return;
}

// Four channels of a token, of which `left` are the layer's.
template <typename T>
__device__ __forceinline__ void put4(T* to, const float (&y)[4], int left) {
  if (left >= 4 && (reinterpret_cast<uintptr_t>(to) & (4 * sizeof(T) - 1)) == 0) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) to[i] = from_f32<T>(y[i]);
  }
}

// HALVES: 1: the warpgroups that take sums out take every second group each, 2: half of the tokens each; HALF:
// fp16 operands, else bf16; UNITS: groups per 128 input channels.
template <int HALVES, bool HALF, int UNITS>
__global__ void __launch_bounds__(kThreads, 1)
    quant_fc_tc_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ TcQuantArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  // 128.0 (bf16) or 1024.0 (fp16), whose last significant bits are worth 1: or-ing a 4-bit number
  // in adds it
  constexpr uint32_t kBias = HALF ? 0x6400u : 0x4300u;
  constexpr int kGroup = kQuantK / UNITS;  // input channels of a unit: a group's share of a tile
  constexpr int kScaleBytes = UNITS * kQuantRows * 4;
  uint8_t* const ring_b = smem;
  const int stage_w = w_stage_bytes(UNITS, a.q.zero != nullptr);
  const int scale_stages = a.stages + kScaleSlack;
  uint8_t* const ring_s = smem + kRingBytes - scale_stages * kScaleBytes;
  uint8_t* const ring_w = ring_s - kWStages * stage_w;
  Bars* const B = reinterpret_cast<Bars*>(smem + kRingBytes);
  uint32_t* const err = a.q.err;
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicOr(err, kErrLayout);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster's CTAs share the input channels of one tile; otherwise tiles cta, cta + ctas, ...
  const int split = static_cast<int>(blockIdx.x) % a.splits;
  const int tile0 = blockIdx.x / a.splits, tile_step = gridDim.x / a.splits;
  const int row_tiles = a.q.no_pad / kQuantRows;
  const int per = (a.q.k_tiles + a.splits - 1) / a.splits;
  const int kt0 = min(split * per, a.q.k_tiles);
  const int n = min(kt0 + per, a.q.k_tiles) - kt0;  // steps (of 128 input channels) of a tile
  const int my_tiles = tile0 < a.tiles ? (a.tiles - tile0 + tile_step - 1) / tile_step : 0;
  const int steps = my_tiles * n;
  const bool joined = a.splits > 1 || a.fold > 1;  // sums that meet in shared memory (one tile a CTA)
  const int piece_bytes = a.cols * kQuantK * 2;     // of a tile and part: [64-channel block][token][128 bytes]
  const int stage_b = a.parts * piece_bytes;
  const uint32_t bars = smem_u32(B);
  const uint32_t ready = bars + offsetof(Bars, ready), done = bars + offsetof(Bars, done);
  const uint32_t full_w = bars + offsetof(Bars, full_w), empty_w = bars + offsetof(Bars, empty_w);
  const uint32_t full_d = bars + offsetof(Bars, full_d), empty_d = bars + offsetof(Bars, empty_d);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&B->ready[i], 1 + 4);
      mbar_init(&B->done[i], 1);
    }
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&B->full_w[i], 1);
      mbar_init(&B->empty_w[i], 4);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&B->full_d[i], 1);
      mbar_init(&B->empty_d[i], HALVES * 4);
    }
    mbar_init(&B->last, 1);
    B->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tensor_map(&tmB);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B->tmem_base)),
                 "r"(static_cast<uint32_t>(kTmemCols)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_base;
  const uint32_t tmem_a = tmem + static_cast<uint32_t>(kSlots / HALVES * a.slot_cols);
  // The groups of a tile's steps, in order, as offsets of the tile's channels in a [groups][no_pad] array (counted, so
  // that the copying threads divide once a tile).  Behind the last group the inputs are 0.
  const int last_group = (a.q.k + a.q.group - 1) / a.q.group - 1, steps_per_group = max(a.q.group / kQuantK, 1);
  struct Groups {
    int64_t at;
    int group, left;
  };
  auto first_group = [&](int rt) {
    const int g = UNITS == 1 ? kt0 / steps_per_group : kt0 * UNITS;
    return Groups{static_cast<int64_t>(min(g, last_group)) * a.q.no_pad + rt * kQuantRows, g,
                  UNITS == 1 ? steps_per_group - (kt0 - g * steps_per_group) : 1};
  };
  auto next_group = [&](Groups& g) {
    if (--g.left == 0) {
      if (g.group++ < last_group) g.at += a.q.no_pad;
      g.left = steps_per_group;
    }
  };

  // The launch has 96 registers a thread, 5 x 96 in all: 40 + 2 x 72 + 2 x 144.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      if (elect_one()) {
        // ---------------- tokens and scales ----------------
        wait_prior_grid();
        int s = 0, ss = 0, issued = 0;
        uint32_t phase = 1;
        const uint32_t bytes = static_cast<uint32_t>(stage_b + kScaleBytes);
        bool ok = true;
        for (int tile = tile0; tile < a.tiles && ok; tile += tile_step) {
          const int rt = tile % row_tiles, token0 = tile / row_tiles * a.cols;
          Groups group = first_group(rt);
          int c = kt0 * kQuantK;
          for (int i = 0; i < n; ++i, c += kQuantK) {
            if (!(ok = wait(done + 8 * s, phase, B, err))) break;
            mbar_expect_tx(&B->ready[s], bytes);
            uint8_t* to = ring_b + s * stage_b;
            for (int p = 0, at = token0; p < a.parts; ++p, to += piece_bytes, at += a.part_rows) {
              tma_load_2d(to, &tmB, &B->ready[s], c, at);
              tma_load_2d(to + a.cols * 128, &tmB, &B->ready[s], c + 64, at);
            }
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
              bulk_load(ring_s + ss * kScaleBytes + u * kQuantRows * 4, a.q.scale + group.at, kQuantRows * 4,
                        &B->ready[s]);
              next_group(group);
            }
            ++issued;
            if (++ss == scale_stages) ss = 0;
            if (++s == a.stages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
        if (*reinterpret_cast<volatile uint32_t*>(&B->abort_flag)) drain(B->ready, a.stages, issued);
      }
    } else if (warp == 1) {
      if (elect_one()) {
        // ---------------- MMAs ----------------
        constexpr int kSteps = kGroup / 16;  // MMAs of a unit and part
        constexpr int kBlockSteps = 4;       // MMAs of a 64-channel block
        const uint32_t idesc = (1u << 4) | (HALF ? 0u : (1u << 7) | (1u << 10)) |
                               (static_cast<uint32_t>(a.cols >> 3) << 17) | (8u << 24);
        const uint32_t desc0 = ((smem_u32(ring_b) & 0x3ffffu) >> 4) | (1u << 16);
        const uint32_t desc_stage = static_cast<uint32_t>(stage_b) >> 4;
        const uint32_t desc_piece = static_cast<uint32_t>(piece_bytes) >> 4;
        const uint32_t desc_block = static_cast<uint32_t>(a.cols) * 8u;
        uint32_t desc = desc0, ready_ph = 0;
        // slot: 2 * stream + turn (streams: every second unit), or turn
        uint32_t turn = 0, empty_ph = 1, stream = 0;
        int s = 0, as = 0;
        bool ok = true;
        for (int i = 0; i < steps && ok; ++i) {
          if (!(ok = wait(ready + 8 * s, ready_ph, B, err))) break;
          const uint32_t a_tmem = tmem_a + static_cast<uint32_t>(as * kACols);
          if (++as == a.a_stages) as = 0;
#pragma unroll
          for (int u = 0; u < UNITS; ++u) {
            const uint32_t slot = HALVES == 2 ? turn : 2u * stream + turn;
            if (!ok || !(ok = wait(empty_d + 8 * slot, empty_ph, B, err))) break;
            tc_fence_after();
            const uint32_t d = tmem + slot * static_cast<uint32_t>(a.slot_cols);
            uint32_t lo = desc;
            for (int p = 0; p < a.parts; ++p, lo += desc_piece) {
#pragma unroll
              for (int k = u * kSteps; k < (u + 1) * kSteps; ++k) {
                const uint32_t b = lo + (k >= kBlockSteps ? desc_block : 0u) + (k % kBlockSteps) * 2u;
                if (k == u * kSteps) mma_ts(d, a_tmem + k * 8, b, idesc, p > 0);
                else mma_ts_add(d, a_tmem + k * 8, b, idesc);
              }
            }
            commit(full_d + 8 * slot);
            if (HALVES == 1) stream ^= 1u;
            if (HALVES == 2 || stream == 0) {
              turn ^= 1u;
              if (turn == 0) empty_ph ^= 1u;
            }
          }
          if (!ok) break;
          commit(done + 8 * s);
          desc += desc_stage;
          if (++s == a.stages) {
            s = 0;
            desc = desc0;
            ready_ph ^= 1u;
          }
        }
        tc_commit(&B->last);
        // (also after giving up: nothing may be in flight when the TMEM is freed)
        const uint64_t t0 = globaltimer();
        while (!mbar_try_suspend(&B->last, 0, 20000u))
          if (globaltimer() - t0 > kTimeoutNs) {
            atomicOr(err, kErrTimeout);
            break;
          }
      }
    } else if (warp == 2) {
      if (elect_one()) {
        // ---------------- codes and zeros ----------------
        int s = 0, issued = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int tile = tile0; tile < a.tiles && ok; tile += tile_step) {
          const int rt = tile % row_tiles;
          const uint8_t* from = reinterpret_cast<const uint8_t*>(a.q.codes) +
                                (static_cast<int64_t>(rt) * a.q.k_tiles + kt0) * kQuantTileBytes;
          Groups group = first_group(rt);
          for (int i = 0; i < n; ++i, from += kQuantTileBytes) {
            if (!(ok = wait(empty_w + 8 * s, phase, B, err))) break;
            ++issued;
            uint8_t* to = ring_w + s * stage_w;
            mbar_expect_tx(&B->full_w[s], static_cast<uint32_t>(stage_w));
            bulk_load(to, from, kQuantTileBytes, &B->full_w[s]);
            if (a.q.zero)
#pragma unroll
              for (int u = 0; u < UNITS; ++u) {
                bulk_load(to + kQuantTileBytes + u * kQuantRows, a.q.zero + group.at, kQuantRows, &B->full_w[s]);
                next_group(group);
              }
            if (++s == kWStages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) drain(B->full_w, kWStages, issued);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------- codes -> operands: steps odd, odd + 2, ... ----------------
    const int odd = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int ws = odd % kWStages, as = odd;
    uint32_t wph = 0;
    int s = odd % a.stages, ds = odd % a.stages;  // of step i and of step i - a_stages, whose place it takes
    uint32_t dph = 0;
    for (int i = odd; i < steps; i += 2) {
      if (!wait_warp(full_w + 8 * ws, wph, B, err)) break;
      const uint8_t* from = ring_w + ws * stage_w + row * 16;
      uint32_t w[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint4 v = *reinterpret_cast<const uint4*>(from + t * kQuantRows * 16);
        w[t][0] = v.x; w[t][1] = v.y; w[t][2] = v.z; w[t][3] = v.w;
      }
      // kBias + zero of the four 32-channel chunks, twice in a word
      uint32_t zz[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t z =
            a.q.zero ? ring_w[ws * stage_w + kQuantTileBytes + (c * UNITS >> 2) * kQuantRows + row] : 8u;
        zz[c] = (kBias | z) * 0x10001u;
      }
      __syncwarp();
      if (elect_one()) arrive(empty_w + 8 * ws);
      ws += 2;
      if (ws >= kWStages) {
        ws -= kWStages;
        wph ^= 1u;
      }
      bool ok = true;
#pragma unroll
      for (int two = 0; two < 2; ++two) {
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            uint32_t p[4];
            decode<HALF>(w[t][2 * two + c], zz[2 * two + c], p);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[c * 16 + t * 4 + i] = p[i];
          }
        if (two == 0) {  // the place is free when the MMAs of step i - a_stages are done
          if (i >= a.a_stages) {
            ok = wait_warp(done + 8 * ds, dph, B, err);
            ds += 2;
            if (ds >= a.stages) {
              ds -= a.stages;
              dph ^= 1u;
            }
          }
          if (!ok) break;
          tc_fence_after();
        }
        st_32x32(tmem_a + lanes + static_cast<uint32_t>(as * kACols + two * 32), v);
      }
      if (!ok) break;
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (elect_one()) arrive(ready + 8 * s);
      s += 2;
      if (s >= a.stages) s -= a.stages;
      as += 2;
      if (as >= a.a_stages) as -= a.a_stages;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    // ---------------- sums of groups -> registers ----------------
    const int stream = (warp - 12) >> 2, row = (warp & 3) * 32 + lane;
    const int half = HALVES == 2 ? a.cols / 2 : a.cols;  // tokens of this stream
    const uint32_t from = tmem + static_cast<uint32_t>(stream * (HALVES == 2 ? half : 2 * a.slot_cols)) +
                          (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int chunks = half / 16;
    bool ok = true;
    uint32_t turn = 0, phase = 0;
    const float* scale = reinterpret_cast<const float*>(ring_s) + row;
    int ss = 0, u = 0;  // of this stream's next unit
    if (HALVES == 1 && stream) {
      if (UNITS == 1) ss = 1;
      else u = 1;
    }
    // units of a tile; with one half, this stream's are those of its parity, counted through all tiles
    const int units = n * UNITS;
    int unit = HALVES == 2 ? 0 : stream;  // this stream's next unit, relative to the tile
    float* const xchg = reinterpret_cast<float*>(a.exchange ? smem + kRingBytes - scale_stages * kScaleBytes -
                                                                   kWStages * stage_w - a.exchange
                                                             : ring_b);
    for (int tile = tile0; tile < a.tiles; tile += tile_step) {
      const int rt = tile % row_tiles;
      const int64_t token0 = static_cast<int64_t>(tile / row_tiles) * a.cols;
      uint64_t acc[kMaxCols / 2];  // pairs of neighbouring tokens, for the packed multiply-add
#pragma unroll
      for (int j = 0; j < kMaxCols / 2; ++j) acc[j] = 0;
      for (; unit < units && ok; unit += HALVES == 2 ? 1 : 2) {
        const uint32_t slot = HALVES == 2 ? turn : 2u * stream + turn;
        if (!(ok = wait_warp(full_d + 8 * slot, phase, B, err))) break;
        tc_fence_after();
        const uint32_t sc = __float_as_uint(scale[(ss * UNITS + u) * kQuantRows]);
        const uint64_t sc2 = pair_u32(sc, sc);
        const uint32_t at = from + turn * static_cast<uint32_t>(a.slot_cols);
        uint32_t v[2][16];
        ld_16(at, v[0]);
#pragma unroll
        for (int c = 0; c < kMaxCols / 16; ++c)
          if (c < chunks) {
            ld_wait(v[c & 1]);
            if (c + 1 < kMaxCols / 16 && c + 1 < chunks) {
              ld_16(at + static_cast<uint32_t>((c + 1) * 16), v[(c + 1) & 1]);
            } else {
              tc_fence_before();
              __syncwarp();
              if (elect_one()) arrive(empty_d + 8 * slot);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[c * 8 + j] = fma2(sc2, pair_u32(v[c & 1][2 * j], v[c & 1][2 * j + 1]), acc[c * 8 + j]);
          }
        turn ^= 1u;
        if (turn == 0) phase ^= 1u;
        u += HALVES == 2 ? 1 : 2;
        while (u >= UNITS) {
          u -= UNITS;
          if (++ss == scale_stages) ss = 0;
        }
      }
      // (having given up, this stream still meets the other one at every barrier)
      unit -= units;
      // one half: the second stream's sums go through shared memory, [token][channel], to the first's threads
      const bool both = HALVES == 1 && !joined;
      if (both && !a.exchange) named_barrier(256);  // (over the token ring: all MMAs that read it are done)
      if (both && stream == 1) {
#pragma unroll
        for (int c = 0; c < kMaxCols / 16; ++c)
          if (c < chunks) {
#pragma unroll
            for (int j = 0; j < 16; ++j) xchg[(c * 16 + j) * kQuantRows + row] = half_of(acc[c * 8 + j / 2], j & 1);
          }
      }
      if (both) named_barrier(256);
      if (ok && !joined && (HALVES == 2 || stream == 0)) {
        // a lane's channel, token by token: a warp writes 32 neighbouring channels
        const int chan = rt * kQuantRows + row;
        const int64_t first = token0 + (HALVES == 2 ? stream * half : 0);
        const int count = static_cast<int>(min(static_cast<int64_t>(half), a.q.rows - first));
        if (chan < a.q.no) {
          const float bias = a.q.bias ? __ldg(a.q.bias + chan) : 0.f;
          auto write = [&](auto* out) {
            using TOut = std::remove_pointer_t<decltype(out)>;
            out += first * a.q.out_stride + chan;
#pragma unroll
            for (int c = 0; c < kMaxCols / 16; ++c)
              if (c * 16 < count) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  float y = half_of(acc[c * 8 + j / 2], j & 1) + bias;
                  if (HALVES == 1) y += xchg[(c * 16 + j) * kQuantRows + row];
                  if (a.q.relu) y = y < 0.f ? 0.f : y;
                  if (c * 16 + j < count) *out = from_f32<TOut>(y);
                  out += a.q.out_stride;
                }
              }
          };
          if (a.out_dtype == BCONV_DTYPE_F32) write(static_cast<float*>(a.q.out));
          else if (a.out_dtype == BCONV_DTYPE_BF16) write(static_cast<__nv_bfloat16*>(a.q.out));
          else write(static_cast<__half*>(a.q.out));
        }
      }
      if (both) named_barrier(256);  // (before the sums of the next tile)
      if (joined) {
        // one tile: this CTA's sums as [token][channel] over the token ring (all MMAs that read it are done), so
        // that a warp adds up and writes 128 channels of a token at a time
        named_barrier(256);
        float* const mine = reinterpret_cast<float*>(ring_b) + (HALVES == 2 ? stream * half * kQuantRows : 0) + row;
        if (HALVES == 2 || stream == 0)
#pragma unroll
          for (int c = 0; c < kMaxCols / 16; ++c)
            if (c < chunks) {
#pragma unroll
              for (int j = 0; j < 16; ++j) mine[(c * 16 + j) * kQuantRows] = half_of(acc[c * 8 + j / 2], j & 1);
            }
        if (HALVES == 1) {  // the other half of the units
          named_barrier(256);
          if (stream == 1)
#pragma unroll
            for (int c = 0; c < kMaxCols / 16; ++c)
              if (c < chunks) {
#pragma unroll
                for (int j = 0; j < 16; ++j) mine[(c * 16 + j) * kQuantRows] += half_of(acc[c * 8 + j / 2], j & 1);
              }
        }
      }
    }
    if (joined) {
      asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (ok && !*reinterpret_cast<volatile uint32_t*>(&B->abort_flag)) {
        // tokens split, split + splits, ... of the tile, the warps taking turns; four channels a lane
        const int rt = tile0 % row_tiles;
        const int64_t token0 = static_cast<int64_t>(tile0 / row_tiles) * a.cols;
        const int w = warp - 12, c0 = rt * kQuantRows + lane * 4;
        float bias[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.q.bias)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c0 + i < a.q.no) bias[i] = __ldg(a.q.bias + c0 + i);
#pragma unroll 1
        for (int j = split + w * a.splits; j < a.cols; j += 8 * a.splits) {
          const int64_t token = token0 + j;
          if (token >= a.q.rows) break;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int f = a.fold - 1; f >= 0; --f) {  // (the smallest part first)
            const uint32_t line = static_cast<uint32_t>((j + f * static_cast<int>(a.q.rows)) * 32 + lane) * 16u;
            float4 p[kMaxSplit];
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i)
              if (i < a.splits)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(p[i].x), "=f"(p[i].y), "=f"(p[i].z), "=f"(p[i].w)
                             : "r"(mapa(ring_b, static_cast<uint32_t>(i)) + line)
                             : "memory");
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i)
              if (i < a.splits) {
                v.x += p[i].x; v.y += p[i].y; v.z += p[i].z; v.w += p[i].w;
              }
          }
          float y[4] = {v.x + bias[0], v.y + bias[1], v.z + bias[2], v.w + bias[3]};
          if (a.q.relu)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = y[i] < 0.f ? 0.f : y[i];
          const int64_t at = token * a.q.out_stride + c0;
          if (a.out_dtype == BCONV_DTYPE_F32) put4(static_cast<float*>(a.q.out) + at, y, a.q.no - c0);
          else if (a.out_dtype == BCONV_DTYPE_BF16) put4(static_cast<__nv_bfloat16*>(a.q.out) + at, y, a.q.no - c0);
          else put4(static_cast<__half*>(a.q.out) + at, y, a.q.no - c0);
        }
      }
    }
  }
  if (joined) {
    __syncwarp();
    // the taking-out warps have passed one cluster barrier already; everyone passes two
    if (warp < 12) asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    cluster_sync();  // no CTA leaves while a peer may still read its part
  }
  allow_next_grid();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(kTmemCols)));
  }
}

// Rows the TMA cannot read as they are into [parts][rows][k_pad] 16-bit elements (k_pad a multiple of
// 64, padding 0): fp32 as three bf16 parts that add up to it, 16-bit types unchanged.
template <typename T, typename T16>
__global__ void quant_fc_stage_kernel(const T* __restrict__ in, int64_t stride, int64_t rows, int k, int k_pad,
                                      T16* __restrict__ out) {
  const int64_t pairs = static_cast<int64_t>(k_pad / 2);
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= rows * pairs) return;
  const int64_t r = i / pairs;
  const int c = static_cast<int>(i - r * pairs) * 2;
  const T zero = from_f32<T>(0.f);
  const T x0 = c < k ? in[r * stride + c] : zero, x1 = c + 1 < k ? in[r * stride + c + 1] : zero;
  uint32_t* to = reinterpret_cast<uint32_t*>(out) + i;
  if constexpr (sizeof(T) == 4) {
    uint32_t hi, mid, lo;
    split3_bf16x2(x0, x1, hi, mid, lo);
    const int64_t part = rows * pairs;
    to[0] = hi;
    to[part] = mid;
    to[2 * part] = lo;
  } else {
    *to = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&x0)) |
          (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&x1)) << 16);
  }
}

struct Plan {
  int halves, cols, stages, splits, exchange;
  int64_t tiles;
};

// Tokens per CTA and CTAs per tile, for `rows` rows of `parts` parts (one_tile: all rows in one tile).  A CTA's time
// for 128 input channels is about max(4 tokens, kFloor) cycles: the MMAs, or reading and decoding 8 KB of codes.  Token counts that fill whole waves of
// CTAs win over large tiles with a ragged last wave; leftover SMs share the input channels.
Plan plan_for(const QuantFcArgs& q, int64_t rows, int parts, int most_halves, bool one_tile) {
  constexpr int kFloor = 600;
  const int sms = current_sm_count();
  const int row_tiles = q.no_pad / kQuantRows;
  const int most = parts == 1 ? kMaxCols : 64;  // (the parts' stages take the space)
  Plan best{};
  double best_cost = 1e300;
  for (int halves = 1; halves <= most_halves; ++halves) {
    const int64_t least = ceil_div(rows, most * halves);
    for (int64_t t = least; t < least + (one_tile ? 1 : 6); ++t) {
      const int cols = round_up(static_cast<int>(ceil_div(rows, t)), 16 * halves);
      const int64_t tiles = ceil_div(rows, cols) * row_tiles;
      int splits = 1;
      while (splits < kMaxSplit && tiles * splits * 2 <= sms && q.k_tiles >= splits * 4) splits *= 2;
      const double per = std::max(4.0 * cols * parts, static_cast<double>(kFloor));
      const double cost = static_cast<double>(ceil_div(tiles * splits, sms)) *
                          (per * static_cast<double>(ceil_div(q.k_tiles, splits)) + 1000.0 + 8.0 * cols);
      if (cost < best_cost) {
        best_cost = cost;
        best = {halves, cols, 0, splits, 0, tiles};
      }
    }
  }
  const int units = q.group >= kQuantK ? 1 : kQuantK / q.group;
  const int scale = units * kQuantRows * 4;
  best.exchange = best.halves == 1 && best.tiles > sms ? best.cols * kQuantRows * 4 : 0;
  const int left = kRingBytes - kWStages * w_stage_bytes(units, q.zero) - kScaleSlack * scale - best.exchange;
  best.stages = std::min(kMaxStages, left / (parts * best.cols * kQuantK * 2 + scale));
  return best;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

template <int HALVES, bool HALF, int UNITS>
cudaError_t launch(const CUtensorMap& map, const TcQuantArgs& a, int64_t tiles, cudaStream_t s) {
  auto kern = quant_fc_tc_kernel<HALVES, HALF, UNITS>;
  cudaError_t e = allow_smem<quant_fc_tc_kernel<HALVES, HALF, UNITS>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.splits > 1 ? tiles * a.splits : std::min<int64_t>(tiles, current_sm_count())));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.staged ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, map, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

bool quant_fc_tma_reads(const void* in, int64_t in_stride, int k, int in_dtype) {
  return in_dtype != BCONV_DTYPE_F32 && aligned16(in) && in_stride % 8 == 0 && k >= 64 && in_stride < (int64_t{1} << 38);
}

int64_t quant_fc_tc_workspace(int64_t rows, int k, int in_dtype) {
  return (in_dtype == BCONV_DTYPE_F32 ? 3 : 1) * rows * round_up(k, 64) * 2;
}

cudaError_t launch_quant_fc_tc(const QuantFcArgs& q, int in_dtype, int out_dtype, void* workspace, cudaStream_t s) {
  const bool f32 = in_dtype == BCONV_DTYPE_F32, half = in_dtype == BCONV_DTYPE_F16;
  const bool staged = !quant_fc_tma_reads(q.in, q.in_stride, q.k, in_dtype);
  const bool fold = f32 && 3 * q.rows <= kMaxCols && q.no_pad / kQuantRows <= current_sm_count();
  const int parts = f32 && !fold ? 3 : 1;
  const int k_pad = round_up(q.k, 64);
  if (staged) {
    const int64_t n = q.rows * (k_pad / 2);
    const unsigned blocks = static_cast<unsigned>(ceil_div(n, 256));
    if (f32)
      quant_fc_stage_kernel<<<blocks, 256, 0, s>>>(static_cast<const float*>(q.in), q.in_stride, q.rows, q.k, k_pad,
                                                   static_cast<__nv_bfloat16*>(workspace));
    else
      quant_fc_stage_kernel<<<blocks, 256, 0, s>>>(static_cast<const __half*>(q.in), q.in_stride, q.rows, q.k, k_pad,
                                                   static_cast<__half*>(workspace));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const Plan p = fold ? plan_for(q, 3 * q.rows, 1, 1, true) : plan_for(q, q.rows, parts, parts == 1 ? 2 : 1, false);
  TcQuantArgs a{};
  a.q = q;
  a.cols = p.cols;
  // What the accumulators leave of TMEM holds decoded tiles, but no more of them than tokens: step i arrives on
  // the barrier of step i - stages, whose phase must be over.
  a.slot_cols = round_up(p.cols, 32);
  a.a_stages = std::min((kTmemCols - kSlots / p.halves * a.slot_cols) / kACols, p.stages) / 2 * 2;
  a.parts = parts;
  a.fold = fold ? 3 : 1;
  a.part_rows = static_cast<int>(q.rows);
  a.stages = p.stages;
  a.tiles = static_cast<int>(p.tiles);
  a.exchange = p.exchange;
  a.units = q.group >= kQuantK ? 1 : kQuantK / q.group;
  a.splits = p.splits;
  a.out_dtype = out_dtype;
  a.staged = staged;
  if (a.stages < 2 || a.a_stages < 2 || a.cols > kMaxCols * p.halves) return cudaErrorInvalidValue;
  auto enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(staged ? k_pad : q.k),
                              static_cast<cuuint64_t>(f32 ? q.rows * 3 : q.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(staged ? k_pad : q.in_stride) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(p.cols)};
  const cuuint32_t elem[2] = {1, 1};
  if (enc(&map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
          const_cast<void*>(staged ? workspace : q.in), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
      CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const auto with_units = [&](auto halves, auto is_half) {
    constexpr int kHalves = decltype(halves)::value;
    constexpr bool kHalf = decltype(is_half)::value;
    switch (a.units) {
      case 1: return launch<kHalves, kHalf, 1>(map, a, p.tiles, s);
      case 2: return launch<kHalves, kHalf, 2>(map, a, p.tiles, s);
      default: return launch<kHalves, kHalf, 4>(map, a, p.tiles, s);
    }
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (p.halves == 2) return half ? with_units(Two{}, std::true_type{}) : with_units(Two{}, std::false_type{});
  return half ? with_units(One{}, std::true_type{}) : with_units(One{}, std::false_type{});
}

}  // namespace bconv
