// Products of ragged groups of rows (prox_grouped_matmul):
//   out[r][j] = sum_k a[src(r)][k] W_g[j][k]          rows r of group g
//   gated:     (a W_up^T)[r][j] * act((a W_gate^T)[r][j])
// for fp32, bf16 and e4m3 values (the last with one fp32 scale per row and 128
// inputs and one per 128 x 128 block of W).
//
// The matrix cores compute out^T: the weights' rows (channels) are the M side,
// the tokens the N side.  A lane of the 16 x 16 result then holds four
// neighbouring channels of one token, so a token's scale is one register, a
// gated product has up and gate of a channel in the same lane, and stores are
// four channels wide.  K advances by 128 bytes of a row (32 fp32, 64 bf16, 128
// e4m3 values): a tile row in LDS is eight 16-byte chunks, chunk c of row r at
// place c ^ (r % 8), so that the eight rows of a fragment read touch all banks.
// The order of k inside a step does not matter as long as both sides agree, so
// all three types read the same two 16-byte chunks per lane and step.
#include <algorithm>
#include <cmath>

#include "experts_internal.h"
#include "prox_device.h"

namespace prox {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;

struct Fp8Tag {};

// Two 16-byte chunks of a row: what one lane feeds to the matrix cores per step.
struct Frag {
  u32x4_t c[2];
};

template <typename T>
__device__ __forceinline__ f32x4_t mma(const Frag& w, const Frag& x, f32x4_t acc);
template <>
__device__ __forceinline__ f32x4_t mma<Bf16Tag>(const Frag& w, const Frag& x, f32x4_t acc) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w.c[i]),
                                                  __builtin_bit_cast(bf16x8_t, x.c[i]), acc, 0, 0, 0);
  return acc;
}
template <>
__device__ __forceinline__ f32x4_t mma<F32Tag>(const Frag& w, const Frag& x, f32x4_t acc) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4_t a = __builtin_bit_cast(f32x4_t, w.c[i]), b = __builtin_bit_cast(f32x4_t, x.c[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
  }
  return acc;
}
// The e4m3 form, without block scales in the instruction (scale operands 0).
// Of eight neighbouring products the matrix cores cut each off, towards zero, to a
// multiple of 2^(e - 13), e the largest sum of two factors' exponents, subnormal
// codes counting as -6 (measured, both e4m3 instructions alike: results agree with
// that rule to fp32 rounding).  A product of two codes has seven bits, so only those
// more than 2^7 below the largest lose any.  The eights are added in fp32, the
// 128-blocks by one rounded fp32 multiply-add each.  For activations and weights as
// layers have them the cut costs 3e-5 of the result (of its norm; bf16 results are
// rounded by 1.6e-3), far below the codes' own 2^-4, and twice the rate of bf16
// products of the widened codes, so it is taken as it is.
template <>
__device__ __forceinline__ f32x4_t mma<Fp8Tag>(const Frag& w, const Frag& x, f32x4_t acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8_t, w),
                                                          __builtin_bit_cast(i32x8_t, x), acc, 0, 0, 0, 0, 0, 0);
}

typedef __attribute__((address_space(3))) uint8_t* lds_ptr_t;
__device__ __forceinline__ uint32_t lds_offset(void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr_t)(p)));
}

// A copy's LDS address is in m0, a reserved register: the compiler says so at every
// copy, and uses m0 nowhere else in these kernels.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes per lane from memory to LDS at byte `to` + 16 * lane (`to` is
// uniform).  Written out, since behind the builtin the compiler waits for every
// copy under way before it reads any LDS; the copies have no result register,
// and wait_copies_and_meet() stands between them and the reads of what they
// bring.
__device__ __forceinline__ void copy16(const void* src, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(src) : "m0");
}
__device__ __forceinline__ void copy16(const uint8_t* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base)
               : "m0");
}

// 4 bytes per lane, to LDS at `to` + 4 * lane.
__device__ __forceinline__ void copy4(const void* src, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(src) : "m0");
}
#pragma clang diagnostic pop

struct Item {
  int group, row0, rows, channel_tile;  // rows: those of the tile, 1 .. BT
};

// The rows [lo, hi) of a group, inside [0, rows) whatever the offsets say.
__device__ __forceinline__ void group_rows(const GroupedArgs& a, int g, int* lo, int* hi) {
  if (a.offsets == nullptr) {
    *lo = 0;
    *hi = a.rows;
  } else {
    *lo = min(max(a.offsets[g], 0), a.rows);
    *hi = min(max(a.offsets[g + 1], *lo), a.rows);
  }
}

// The (token tile of kTile, channel tile) of this block.  Items run group by group;
// within a group the token tiles run fastest.  Blocks go round the eight XCDs, each
// with an L2 of its own: XCD x takes the x-th eighth of the items, so that the
// blocks that share a group's weights share an L2.  False: no item is left.  (If
// offsets do not ascend, tiles may be left out, but none is outside the buffers.)
template <int kTile>
__device__ __forceinline__ bool find_item(const GroupedArgs& a, int channel_tiles, Item* shared, int* wave_total) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int per = (a.n_groups + nthr - 1) / nthr, g0 = tid * per;  // neighbouring groups of a thread
  const int g1 = min(g0 + per, a.n_groups);
  int mine = 0;
  for (int g = g0; g < g1; ++g) {
    int lo, hi;
    group_rows(a, g, &lo, &hi);
    mine += (hi - lo + kTile - 1) / kTile;
  }
  int before = wave_inclusive_scan_int(mine);
  if ((tid & 63) == 63) wave_total[tid >> 6] = before;
  if (tid == 0) shared->rows = 0;
  __syncthreads();
  before -= mine;
  int total = 0;
  for (int w = 0; w < nthr >> 6; ++w) {
    if (w < (tid >> 6)) before += wave_total[w];
    total += wave_total[w];
  }
  const int64_t items = static_cast<int64_t>(total) * channel_tiles, share = (items + 7) >> 3;
  const int64_t nth = blockIdx.x >> 3, item = (blockIdx.x & 7) * share + nth;
  if (nth >= share || item >= items) return false;
  int64_t rem = item - static_cast<int64_t>(before) * channel_tiles;
  if (rem >= 0 && rem < static_cast<int64_t>(mine) * channel_tiles) {
    for (int g = g0; g < g1; ++g) {
      int lo, hi;
      group_rows(a, g, &lo, &hi);
      const int tiles = (hi - lo + kTile - 1) / kTile;
      if (rem < static_cast<int64_t>(tiles) * channel_tiles) {
        const int r = static_cast<int>(rem), m = r % tiles;  // below the launch's grid
        *shared = {g, lo + m * kTile, min(kTile, hi - lo - m * kTile), r / tiles};
        break;
      }
      rem -= static_cast<int64_t>(tiles) * channel_tiles;
    }
  }
  __syncthreads();
  return shared->rows > 0;
}

__device__ __forceinline__ Item uniform(const Item& i) {
  return {__builtin_amdgcn_readfirstlane(i.group), __builtin_amdgcn_readfirstlane(i.row0),
          __builtin_amdgcn_readfirstlane(i.rows), __builtin_amdgcn_readfirstlane(i.channel_tile)};
}

// The gate's activation.  Both are z times a logistic function, z / (1 + e^-y):
// y = z, and for the tanh form of GELU y = 2 sqrt(2/pi) (z + 0.044715 z^3), as
// (1 + tanh(y / 2)) / 2 is that function of y.  Results of 16 bits take the
// hardware's exponential and reciprocal: with the rounded argument they are off
// by at most |y| 2^-23 relative, below 2^-16 while e^-y counts at all.
template <int kOut>
__device__ __forceinline__ float gate(float z, int act) {
  if constexpr (kOut == PROX_F32) {
    return gate_act(z, act);
  } else {
    const float y = act == PROX_ACT_SILU ? z : 1.5957691216057308f * (z + 0.044715f * z * z * z);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y * -1.4426950408889634f));
  }
}

// kCount neighbouring results from channel j on into the row of out at q; `left`
// of them exist.  Rows of out need their element's alignment only: the hardware
// takes wide stores at any address.
template <int kOut, int kCount>
__device__ __forceinline__ void store_results(uint8_t* q, int j, const float (&v)[kCount], int left) {
  if constexpr (kOut == PROX_F32) {
    typedef __attribute__((ext_vector_type(4), aligned(4))) float vec_t;
    float* p = reinterpret_cast<float*>(q) + j;
    if (left >= kCount) {
#pragma unroll
      for (int h = 0; h < kCount; h += 4)
        *reinterpret_cast<vec_t*>(p + h) = vec_t{v[h], v[h + 1], v[h + 2], v[h + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < kCount; ++i)
        if (i < left) p[i] = v[i];
    }
  } else {
    typedef __attribute__((ext_vector_type(kCount), aligned(2))) __bf16 vec_t;
    __bf16* p = reinterpret_cast<__bf16*>(q) + j;
    vec_t b;
#pragma unroll
    for (int i = 0; i < kCount; ++i) b[i] = (__bf16)v[i];
    if (left >= kCount) {
      *reinterpret_cast<vec_t*>(p) = b;
    } else {
#pragma unroll
      for (int i = 0; i < kCount; ++i)
        if (i < left) p[i] = b[i];
    }
  }
}

constexpr uint32_t kWidePart = 32 * (8 * 16 + 4) * 4;  // wide kernel: LDS of a wave's results, two token fragments

// Waits until at most kLeft of this wave's memory-to-LDS copies are under way,
// and for its LDS reads, then for the other waves of the block.
template <int kLeft>
__device__ __forceinline__ void wait_copies_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

// The row of a for row r of the tile (rows past the tile's last repeat it), or
// -1 for a row index outside a.
__device__ __forceinline__ int source_row(const GroupedArgs& a, const Item& it, int r) {
  r = it.row0 + min(r, it.rows - 1);
  const int src = a.row_index ? a.row_index[r] : r;
  return src < a.a_rows ? src : -1;
}

// One lane's share of the copies that bring a step of a tile (BT tokens, BC weight
// rows, 128 bytes of k) into LDS: weight rows first, then tokens, then (fp8)
// scales.  A copy of a wave is eight rows; lane l brings the chunk at place l % 8
// of row l / 8.  Rows past the last token or channel of the tile repeat a row that
// exists; their results are not stored.
template <bool kGated, bool kFp8, int BT, int BC, int kWaves>
struct TileCopies {
  static constexpr int NW = BC / 8 / kWaves, NX = BT / 8 / kWaves, kCount = NW + NX + (kFp8 ? 1 : 0);
  static constexpr uint32_t kScales = (BC + BT) * 128;  // their place in a buffer
  static constexpr uint32_t kBuffer = kScales + (kFp8 ? kWaves * 256 : 0);
  // fp8: wave i < kTokenWaves brings the scales of 64 tokens, the next wave those
  // of the channels (kBlocks blocks of 128, up then gate); lanes and waves
  // without a scale repeat another
  static constexpr int kTokenWaves = (BT + 63) / 64, kBlocks = BC / (kGated ? 256 : 128) + 1;
  static_assert(NW * 8 * kWaves == BC && NX * 8 * kWaves == BT, "whole copies");
  static_assert(!kFp8 || kTokenWaves < kWaves, "a wave is left for the channels' scales");

  // uniform: the tile's first channel in the matrix that copy i takes rows of, for
  // even and odd i (sixteens of rows are up and gate in turn, so with four or more
  // waves all copies of a wave take the same one)
  const uint8_t *w_even, *w_odd;
  uint32_t woff[NW];             // below 2^31: at most 256 rows of less than 2^23 bytes
  const uint8_t* xsrc[NX];
  const float* scale;
  int kbytes, chunk, wave;

  // *outside (LDS, 0 before): set if a row index of the tile is outside a.
  __device__ __forceinline__ void init(const GroupedArgs& a, const Item& it, int c0, int wave_, int lane, int* outside) {
    const int crow = lane >> 3;
    chunk = ((lane & 7) ^ crow) * 16;
    wave = wave_;
    kbytes = a.kbytes;
    const int64_t first = it.group * a.w_group + c0 * a.w_stride;
    const uint8_t* const up = a.w + first;
    const uint8_t* const gate = kGated ? a.w_gate + first : up;
    static_assert(kWaves == 2 || kWaves % 4 == 0, "copies take up or gate rows by wave, or in turn");
    w_even = kWaves > 2 && (wave >> 1 & 1) ? gate : up;
    w_odd = kWaves > 2 ? w_even : gate;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int r = (i * kWaves + wave) * 8 + crow;
      const int j = min(kGated ? (r >> 5) * 16 + (r & 15) : r, a.n - 1 - c0);
      woff[i] = static_cast<uint32_t>(j) * static_cast<uint32_t>(a.w_stride) + chunk;
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int src = source_row(a, it, (i * kWaves + wave) * 8 + crow);
      if (src < 0) *outside = 1;
      xsrc[i] = a.a + max(src, 0) * a.a_stride + chunk;
    }
    scale = nullptr;
    if constexpr (kFp8) {
      if (wave < kTokenWaves) {
        scale = a.a_scale + static_cast<int64_t>(max(source_row(a, it, wave * 64 + lane), 0)) * a.kblocks;
      } else {
        const int block = min(c0 / kScaleBlock + lane % kBlocks, a.nblocks - 1);
        scale = (kGated && (lane / kBlocks & 1) ? a.w_gate_scale : a.w_scale) +
                (static_cast<int64_t>(it.group) * a.nblocks + block) * a.kblocks;
      }
    }
  }

  // This lane's offset for the step at byte kb.  Chunks past the end of k (in the
  // last step only) repeat the step's first one; the products take zeros there.
  __device__ __forceinline__ int offset(int kb) const { return kb + chunk < kbytes ? kb : kb - chunk; }

  // Copy i of the step at kb (off: offset(kb)) into the buffer at LDS byte `to`.
  __device__ __forceinline__ void go(int i, int kb, int off, uint32_t to) const {
    if (i < NW) {
      copy16((i & 1) ? w_odd : w_even, woff[i] + off, to + (i * kWaves + wave) * 1024);
    } else if (i < NW + NX) {
      copy16(xsrc[i - NW] + off, to + BC * 128 + ((i - NW) * kWaves + wave) * 1024);
    } else if constexpr (kFp8) {
      copy4(scale + (kb >> 7), to + kScales + wave * 256);
    }
  }
};

// The two 16-byte chunks of this lane's row in a fragment at p.
struct Places {
  int row, quad, place[2];
  __device__ __forceinline__ explicit Places(int lane)
      : row(lane & 15), quad(lane >> 4), place{((lane >> 4) ^ (lane & 7)) << 4, ((4 + (lane >> 4)) ^ (lane & 7)) << 4} {}
  __device__ __forceinline__ Frag read(const uint8_t* p) const {
    Frag r;
    r.c[0] = *reinterpret_cast<const u32x4_t*>(p + place[0]);
    r.c[1] = *reinterpret_cast<const u32x4_t*>(p + place[1]);
    return r;
  }
};

// The wave's results, FC x 16 weight rows by FT x 16 tokens, to out.  They go
// through the wave's own part of LDS, TP token fragments at a time, so that a row
// of out is written in whole lines and the activation is one short loop (held in
// registers it is unrolled to 40 KB of code, which every CU first has to fetch).
// first: the wave's first channel; token_row(t): the tile's row of fragment t;
// zeros: there are row indices outside a in the tile, whose results are zero.
// WK: that many waves, `group` the number of this one, hold parts of the same
// results (each of a share of k), `apart` floats from part to part; they are added
// up here, in the order of the groups, and the waves share the rows.
template <bool kGated, int kOut, int FC, int FT, int TP, int WK, typename Rows>
__device__ __forceinline__ void write_results(const GroupedArgs& a, const Item& it, const f32x4_t (&acc)[FC][FT],
                                              float* part, int group, int apart, int lane, int first, bool zeros,
                                              Rows token_row) {
  constexpr int kStride = FC * 16 + 4;                 // floats per token: rows four banks apart
  constexpr int kChannels = FC * (kGated ? 8 : 16);    // results per token
  constexpr int kLanes = kChannels / 8, kPer = 64 / kLanes;  // lanes of a token, tokens at a time
  static_assert(WK == 1 || TP == FT, "the groups meet once");
  const int row = lane & 15, quad = lane >> 4;
  const int slot = lane / kLanes, j0 = lane % kLanes * 8;
  const int left = a.n - first - j0;  // results that exist from this lane's first on
#pragma unroll
  for (int t0 = 0; t0 < FT; t0 += TP) {
#pragma unroll
    for (int t = t0; t < t0 + TP; ++t)
#pragma unroll
      for (int f = 0; f < FC; ++f)
        *reinterpret_cast<f32x4_t*>(part + group * apart + ((t - t0) * 16 + row) * kStride + f * 16 + quad * 4) =
            acc[f][t];
    if constexpr (WK > 1) __syncthreads();
#pragma unroll 1
    for (int i = slot + group * kPer; i < TP * 16; i += kPer * WK) {
      const int r = token_row(t0 + (i >> 4)) + (i & 15);
      if (r >= it.rows || left <= 0) continue;
      // a channel's up and gate are sixteen rows apart
      const float* p = part + i * kStride + (kGated ? (j0 >> 4) * 32 + (j0 & 15) : j0);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = p[e];
      for (int g = 1; g < WK; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += p[g * apart + e];
      if constexpr (kGated) {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = p[16 + e];
        for (int g = 1; g < WK; ++g)
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] += p[g * apart + 16 + e];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= gate<kOut>(z[e], a.act);
      }
      if (zeros && source_row(a, it, r) < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      }
      uint8_t* q = a.out + (static_cast<int64_t>(it.row0) + r) * a.out_stride;
      store_results<kOut, 8>(q, first + j0, v, left);
    }
  }
}

// One block: BT tokens x BC weight rows (gated: BC / 2 channels, up and gate in
// turn by sixteen rows), WK groups of WC x WT waves, S LDS buffers a group.  The
// groups take the steps of k in turn: where a launch has too few blocks to fill
// the chip, a block's time is its number of steps, each of which costs a latency.
// While a group multiplies a step, the copies of its next S - 1 are under way.
// (At least two waves per SIMD: with more registers the compiler moves the sums
// between the two register files in every step.)
template <typename T, bool kGated, int kOut, int BT, int BC, int WT, int WC, int WK, int S>
__global__ void __launch_bounds__(64 * WT * WC * WK, 2) tile_kernel(GroupedArgs a) {
  constexpr int kWaves = WT * WC, FC = BC / 16 / WC, FT = BT / 16 / WT;  // fragments of 16 per wave
  constexpr bool kFp8 = std::is_same<T, Fp8Tag>::value;
  typedef TileCopies<kGated, kFp8, BT, BC, kWaves> Copies;
  static_assert(FC * 16 * WC == BC && FT * 16 * WT == BT, "tile");
  static_assert(FC <= 8 && 128 % (FC * 16) == 0, "a wave's channels lie in one scale block");
  static_assert(!kGated || FC % 2 == 0, "up and gate of a channel belong to one wave");
  constexpr uint32_t kBuffer = Copies::kBuffer, kCopies = Copies::kCount;
  constexpr int TP = FT < 2 || WK > 1 ? FT : 2;            // token fragments written at a time
  constexpr uint32_t kPart = TP * 16 * (FC * 16 + 4) * 4;  // LDS of a wave's results
  constexpr uint32_t kLds = WK * (S * kBuffer > kWaves * kPart ? S * kBuffer : kWaves * kPart);
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  __shared__ Item s_item;
  __shared__ int s_total[kWaves * WK], s_outside;
  if (threadIdx.x == 0) s_outside = 0;  // find_item's barrier stands before its use
  const int chan_per_tile = kGated ? BC / 2 : BC;
  const int channel_tiles = (a.n + chan_per_tile - 1) / chan_per_tile;
  if (!find_item<BT>(a, channel_tiles, &s_item, s_total)) return;
  const Item it = uniform(s_item);
  const int lane = threadIdx.x & 63;
  const int number = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = number / kWaves, wave = number % kWaves;
  const int wc = wave / WT, wt = wave % WT;  // this wave's share of the channels and of the tokens
  const int c0 = it.channel_tile * chan_per_tile;
  const int first = c0 + wc * FC * (kGated ? 8 : 16);
  Copies copies;
  copies.init(a, it, c0, wave, lane, &s_outside);
  const Places at(lane);
  uint8_t* const mine = lds + group * (S * kBuffer);  // the group's buffers
  const uint32_t lds0 = lds_offset(mine);
  // the block of 128 channels that this wave's lie in, from the tile's first on
  const int block = first / kScaleBlock - c0 / kScaleBlock;

  f32x4_t acc[FC][FT];
#pragma unroll
  for (int f = 0; f < FC; ++f)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[f][t] = f32x4_t{0, 0, 0, 0};

  // Multiplies the step in buffer `from`, and meanwhile (more) issues the copies
  // of the step at next_kb into `to`, a few between the products.
  const auto multiply = [&](auto more, auto last, int kb, uint32_t from, int next_kb, uint32_t to) {
    const uint8_t* pw = mine + from + (wc * FC * 16 + at.row) * 128;
    const uint8_t* px = mine + from + BC * 128 + (wt * FT * 16 + at.row) * 128;
    const auto read = [&](const uint8_t* p) {
      Frag r = at.read(p);
      if constexpr (decltype(last)::value) {  // chunks past the end of k count as zeros
        if (kb + at.quad * 16 >= a.kbytes) r.c[0] = u32x4_t{0, 0, 0, 0};
        if (kb + at.quad * 16 + 64 >= a.kbytes) r.c[1] = u32x4_t{0, 0, 0, 0};
      }
      return r;
    };
    Frag xf[FT], wf[2];
    wf[0] = read(pw);
#pragma unroll
    for (int t = 0; t < FT; ++t) xf[t] = read(px + t * 2048);
    float xscale[FT], ws_up = 0.f, ws_gate = 0.f;
    f32x4_t part[2][FT];  // fp8: a fragment's products, scaled and added one fragment later
    if constexpr (kFp8) {
      const float* ps = reinterpret_cast<const float*>(mine + from + Copies::kScales);
#pragma unroll
      for (int t = 0; t < FT; ++t) xscale[t] = ps[(wt * FT + t) * 16 + at.row];
      ws_up = ps[Copies::kTokenWaves * 64 + block];
      ws_gate = kGated ? ps[Copies::kTokenWaves * 64 + Copies::kBlocks + block] : ws_up;
      if (WK > 1 && decltype(last)::value && kb >= a.kbytes) {  // no step, no scales
#pragma unroll
        for (int t = 0; t < FT; ++t) xscale[t] = 0.f;
        ws_up = ws_gate = 0.f;
      }
    }
    const auto add = [&](int f) {
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        const float sc = xscale[t] * (kGated && (f & 1) ? ws_gate : ws_up);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(part[f & 1][t][i], sc, acc[f][t][i]);
      }
    };
    const int off = copies.offset(next_kb);
#pragma unroll
    for (int f = 0; f < FC; ++f) {
      // the next channels' fragment is read while this one is multiplied
      if (f + 1 < FC) wf[(f + 1) & 1] = read(pw + (f + 1) * 2048);
      if constexpr (decltype(more)::value) {
#pragma unroll
        for (int i = f * kCopies / FC; i < (f + 1) * kCopies / FC; ++i) copies.go(i, next_kb, off, lds0 + to);
      }
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        if constexpr (kFp8) part[f & 1][t] = mma<T>(wf[f & 1], xf[t], f32x4_t{0, 0, 0, 0});
        else acc[f][t] = mma<T>(wf[f & 1], xf[t], acc[f][t]);
      }
      if constexpr (kFp8) {
        if (f > 0) {
          add(f - 1);
          // a matrix instruction, then the four sums that fit beside it
#pragma unroll
          for (int t = 0; t < FT; ++t) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kFp8) add(FC - 1);
  };
  const int steps = (a.kbytes + 127) / 128;
  const auto copy = [&](int step, uint32_t to) {
    const int kb = step * 128, off = copies.offset(kb);
#pragma unroll
    for (int c = 0; c < static_cast<int>(kCopies); ++c) copies.go(c, kb, off, lds0 + to);
  };
  uint32_t now = 0, next = 0;  // the buffers of this step and of the next copy
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (i * WK + group < steps) copy(i * WK + group, next);
    next += kBuffer;
  }
  const auto advance = [&] {
    next = next == (S - 1) * kBuffer ? 0 : next + kBuffer;
    now = now == (S - 1) * kBuffer ? 0 : now + kBuffer;
  };
  // rounds of one step a group; as long as every group has a step to copy
  int round = 0;
  for (; (round + S) * WK <= steps; ++round) {
    const int step = round * WK + group, then = step + (S - 1) * WK;
    // this step's copies are done when only those of the later steps are left
    wait_copies_and_meet<(S - 2) * kCopies>();
    multiply(std::true_type{}, std::false_type{}, step * 128, now, then * 128, next);
    advance();
  }
  for (; (round + 1) * WK < steps; ++round) {
    const int step = round * WK + group, then = step + (S - 1) * WK;
    wait_copies_and_meet<0>();
    if (then < steps) copy(then, next);
    multiply(std::false_type{}, std::false_type{}, step * 128, now, 0, 0);
    advance();
  }
  // the last round: a group without a step multiplies zeros
  wait_copies_and_meet<0>();
  multiply(std::false_type{}, std::true_type{}, (round * WK + group) * 128, now, 0, 0);
  wait_copies_and_meet<0>();  // every wave has read its last step
  write_results<kGated, kOut, FC, FT, TP, WK>(a, it, acc, reinterpret_cast<float*>(lds + wave * kPart), group,
                                              kWaves * kPart / 4, lane, first, s_outside != 0,
                                              [&](int t) { return (wt * FT + t) * 16; });
}

// Many rows per group: one block computes 256 tokens x 256 weight rows (gated:
// 128 channels, up and gate in turn by sixteen rows) with eight waves of 64
// tokens x 128 weight rows, from two LDS buffers of one step each.  A step has two
// meeting points of the waves: at the first, the tokens and the lower half of
// every wave's channels have been read, at the second the upper half; each part
// is overwritten with the copies of the step after next as soon as it is free.
// So a copy has one and a half steps to arrive, and a wait leaves a whole step's
// copies under way (one meeting per step and one step of distance: 5 to 10 %
// slower).  After the second meeting the first fragments of the next step are read
// under the last products of this one.
// The waves take the token fragments in turn, so that a tile of at most 128
// tokens (FT = 2) costs every wave half the products.
template <typename T, bool kGated, int kOut, int FT>
__device__ __forceinline__ void wide_tile(const GroupedArgs& a, const Item& it, uint8_t* lds, int* outside, int c0) {
  constexpr int BT = FT * 64, BC = 256, WT = 4, kWaves = 8, FC = 8;
  constexpr bool kFp8 = std::is_same<T, Fp8Tag>::value;
  typedef TileCopies<kGated, kFp8, BT, BC, kWaves> Copies;
  constexpr uint32_t kBuffer = Copies::kBuffer;
  constexpr int kCopies = Copies::kCount, NW = Copies::NW;
  static_assert(NW == 4, "copies 0 and 2 of the channels are the lower halves");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wc = wave / WT, wt = wave % WT;  // this wave's share of the channels and of the tokens
  const int first = c0 + wc * FC * (kGated ? 8 : 16);
  Copies copies;
  copies.init(a, it, c0, wave, lane, outside);
  const Places at(lane);
  const uint32_t lds0 = lds_offset(lds);
  const int block = first / kScaleBlock - c0 / kScaleBlock;  // this wave's block of 128 channels in the tile

  f32x4_t acc[FC][FT];
#pragma unroll
  for (int f = 0; f < FC; ++f)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[f][t] = f32x4_t{0, 0, 0, 0};

  const uint8_t* const pw = lds + (wc * FC * 16 + at.row) * 128;
  const uint8_t* const px = lds + BC * 128 + (wt * 16 + at.row) * 128;
  Frag xf[FT], wf[2];  // at the start of a step: its tokens and its first channels
  // Multiplies the step in buffer `from` (the next one is in `then`); more: the
  // step after that one is copied into `from`.
  const auto multiply = [&](auto more, auto last, int kb, uint32_t from, uint32_t then) {
    constexpr bool kMore = decltype(more)::value, kLast = decltype(last)::value;
    const bool out0 = kb + at.quad * 16 >= a.kbytes, out1 = kb + at.quad * 16 + 64 >= a.kbytes;
    const auto cut = [&](Frag& r) {  // chunks past the end of k count as zeros
      if constexpr (kLast) {
        if (out0) r.c[0] = u32x4_t{0, 0, 0, 0};
        if (out1) r.c[1] = u32x4_t{0, 0, 0, 0};
      }
    };
    cut(wf[0]);
#pragma unroll
    for (int t = 0; t < FT; ++t) cut(xf[t]);
    float xscale[FT], ws_up = 0.f, ws_gate = 0.f;
    f32x4_t part[4];  // fp8: products, scaled and added three matrix instructions later
    if constexpr (kFp8) {
      const float* ps = reinterpret_cast<const float*>(lds + from + Copies::kScales);
#pragma unroll
      for (int t = 0; t < FT; ++t) xscale[t] = ps[(t * WT + wt) * 16 + at.row];
      ws_up = ps[Copies::kTokenWaves * 64 + block];
      ws_gate = kGated ? ps[Copies::kTokenWaves * 64 + Copies::kBlocks + block] : ws_up;
    }
    const auto add = [&](int n) {  // the n-th instruction's
      const int f = n / FT, t = n % FT;
      const float sc = xscale[t] * (kGated && (f & 1) ? ws_gate : ws_up);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(part[n & 3][i], sc, acc[f][t][i]);
    };
    const int next_kb = kb + 256, off = kMore ? copies.offset(next_kb) : 0;
#pragma unroll
    for (int f = 0; f < FC; ++f) {
      if (f == FC / 2 - 1) {  // this step's upper half has come; its tokens and lower half are read
        wait_copies_and_meet<kLast ? 0 : kCopies>();
      } else if (f == FC - 1 && !kLast) {  // the next step's lower part has come; the upper half is read
        wait_copies_and_meet<kMore ? kCopies : 2>();
      }
      // the next channels' fragment is read while this one is multiplied
      if (f + 1 < FC) {
        wf[(f + 1) & 1] = at.read(pw + from + (f + 1) * 2048);
        cut(wf[(f + 1) & 1]);
      } else if constexpr (!kLast) {
        wf[0] = at.read(pw + then);
      }
      if constexpr (kMore) {
        // lower part: spread over three fragments' products (issued at once the
        // copies hold up the reads); upper half
        if (f == FC / 2 - 1) {
          copies.go(0, next_kb, off, lds0 + from);
          copies.go(2, next_kb, off, lds0 + from);
        } else if (f == FC / 2 || f == FC / 2 + 1) {
#pragma unroll
          for (int i = NW; i < kCopies; ++i)
            if ((i - NW >= 2) == (f > FC / 2)) copies.go(i, next_kb, off, lds0 + from);
        } else if (f == FC - 1) {
          copies.go(1, next_kb, off, lds0 + from);
          copies.go(3, next_kb, off, lds0 + from);
        }
      }
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        if constexpr (kFp8) {
          const int n = f * FT + t;
          part[n & 3] = mma<T>(wf[f & 1], xf[t], f32x4_t{0, 0, 0, 0});
          if (n >= 3) add(n - 3);
          // a matrix instruction, then the sums that fit beside it
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        } else {
          acc[f][t] = mma<T>(wf[f & 1], xf[t], acc[f][t]);
        }
        if constexpr (!kLast) {
          if (f == FC - 1) xf[t] = at.read(px + then + t * (WT * 2048));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kFp8) {
#pragma unroll
      for (int n = FC * FT - 3; n < FC * FT; ++n) add(n);
    }
  };
  // the first two steps, in the order of the waits: lower parts, then upper halves
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s * 128 < a.kbytes) {
      const int off = copies.offset(s * 128);
      const uint32_t to = lds0 + s * kBuffer;
      copies.go(0, s * 128, off, to);
      copies.go(2, s * 128, off, to);
#pragma unroll
      for (int i = NW; i < kCopies; ++i) copies.go(i, s * 128, off, to);
      copies.go(1, s * 128, off, to);
      copies.go(3, s * 128, off, to);
    }
  }
  if (128 < a.kbytes) wait_copies_and_meet<kCopies + 2>();
  else wait_copies_and_meet<2>();
  wf[0] = at.read(pw);
#pragma unroll
  for (int t = 0; t < FT; ++t) xf[t] = at.read(px + t * (WT * 2048));
  uint32_t now = 0;  // this step's buffer
  int kb = 0;
  for (; kb + 256 < a.kbytes; kb += 128) {
    multiply(std::true_type{}, std::false_type{}, kb, now, now ^ kBuffer);
    now ^= kBuffer;
  }
  if (kb + 128 < a.kbytes) {
    multiply(std::false_type{}, std::false_type{}, kb, now, now ^ kBuffer);
    kb += 128;
    now ^= kBuffer;
  }
  multiply(std::false_type{}, std::true_type{}, kb, now, 0);
  wait_copies_and_meet<0>();  // every wave has read its last step
  write_results<kGated, kOut, FC, FT, 2, 1>(a, it, acc, reinterpret_cast<float*>(lds + wave * kWidePart), 0, 0, lane,
                                            first, *outside != 0, [&](int t) { return (t * WT + wt) * 16; });
}

template <typename T, bool kGated, int kOut>
__global__ void __launch_bounds__(512) wide_kernel(GroupedArgs a) {
  constexpr uint32_t kBuffers = 2 * TileCopies<kGated, std::is_same<T, Fp8Tag>::value, 256, 256, 8>::kBuffer;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBuffers > 8 * kWidePart ? kBuffers : 8 * kWidePart];
  __shared__ Item s_item;
  __shared__ int s_total[8], s_outside;
  if (threadIdx.x == 0) s_outside = 0;  // find_item's barrier stands before its use
  const int chan_per_tile = kGated ? 128 : 256;
  const int channel_tiles = (a.n + chan_per_tile - 1) / chan_per_tile;
  if (!find_item<256>(a, channel_tiles, &s_item, s_total)) return;
  const Item it = uniform(s_item);
  if (it.rows > 128) wide_tile<T, kGated, kOut, 4>(a, it, lds, &s_outside, it.channel_tile * chan_per_tile);
  else wide_tile<T, kGated, kOut, 2>(a, it, lds, &s_outside, it.channel_tile * chan_per_tile);
}

// Blocks of a launch: at least the items that offsets can make.
int64_t grid_blocks(const GroupedArgs& a, int bt, int channels) {
  const int64_t tiles = a.rows / bt + std::min(a.n_groups, a.rows);
  return (tiles * ((a.n + channels - 1) / channels) + 7) / 8 * 8;
}

template <typename T, bool kGated, int kOut>
hipError_t launch_wide(const GroupedArgs& a, hipStream_t s) {
  const int64_t grid = grid_blocks(a, 256, kGated ? 128 : 256);
  if (!grid_fits(grid, 512)) return hipErrorInvalidConfiguration;
  wide_kernel<T, kGated, kOut><<<dim3(static_cast<unsigned>(grid)), dim3(512), 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, bool kGated, int kOut, int BT, int BC, int WT, int WC, int WK, int S>
hipError_t launch_tile(const GroupedArgs& a, hipStream_t s) {
  const int64_t grid = grid_blocks(a, BT, kGated ? BC / 2 : BC);
  if (!grid_fits(grid, 64 * WT * WC * WK)) return hipErrorInvalidConfiguration;
  tile_kernel<T, kGated, kOut, BT, BC, WT, WC, WK, S>
      <<<dim3(static_cast<unsigned>(grid)), dim3(64 * WT * WC * WK), 0, s>>>(a);
  return hipGetLastError();
}

// Which kernel.  A block's time is its rounds of steps times the time of one: a
// latency while the launch leaves CUs idle, and a share of the CU once there are
// several blocks to each.  The shape with the smallest estimate,
//   rounds * max(latency, blocks / CUs * cost),
// is taken.  What the host knows is rows, groups and sizes, not how the rows
// spread: a group of m rows on average counts as m / tokens + 1/2 tiles.  The
// figures (us a step) were fitted on MI355X over 920 products of 1 to 64 groups, 1
// to 1024 rows a group, n 256 to 12288 and k 256 to 12288.  With the present stores,
// over 888 such products, the choice is 1.6 % (bf16), 1.4 % (fp8) and 1.8 % (fp32)
// behind the best of these shapes in the mean, 5 % at the ninetieth hundredth, and
// 33, 37 and 43 % at worst (fp32: 16 groups of 65 rows, n 1500, k 1008: 64 x 128 74.5
// us, 32 x 32 in two K groups 52).  For example (bf16, us): 64 groups, n 2048, k 1024,
// m 256: wide 115, 64 x 128 tiles 143; m 16: 32 x 64 55, wide 61; one group, n = k =
// 4096, m 128: 32 x 32 in two K groups 17, 32 x 64 in one 19.
enum Shape { kWide, k128x256, k64x128, k64x64, k32x64, k32x32by2, k32x32by4, kShapes };
struct ShapeTime {
  int tokens, channels, groups;  // a block's tile, and how many groups of waves share k
  float latency, cost;
};
constexpr ShapeTime kTimes[kShapes] = {
    {256, 256, 1, 2.0f, 2.4f},  {128, 256, 1, 1.2f, 1.6f},  {64, 128, 1, 0.45f, 0.51f}, {64, 64, 1, 0.30f, 0.29f},
    {32, 64, 1, 0.26f, 0.23f},  {32, 32, 2, 0.25f, 0.25f},  {32, 32, 4, 0.43f, 0.71f}};
// fp32 products run at 256 flops per clock and CU at most, which 64 x 128 tiles reach
// to three quarters (16 groups of 1024 rows, n = k = 1024: matrix cores 72 % busy, 307
// us, 112 TFLOP/s; one group of 4096 rows, n = k = 2048: 126 of the 153 of a large
// library product); the two large shapes are not built for them
constexpr ShapeTime kTimesF32[kShapes] = {
    {0, 0, 0, 0, 0},            {0, 0, 0, 0, 0},            {64, 128, 1, 1.12f, 1.35f}, {64, 64, 1, 0.61f, 0.72f},
    {32, 64, 1, 0.61f, 0.50f},  {32, 32, 2, 0.47f, 0.43f},  {32, 32, 4, 0.68f, 0.89f}};

Shape choose_shape(const GroupedArgs& a, int cus) {
  const ShapeTime* times = a.wdtype == PROX_F32 ? kTimesF32 : kTimes;
  const int live = std::min(a.n_groups, a.rows);  // groups that can have rows
  const double n = static_cast<double>(a.n) * (a.w_gate ? 2 : 1);
  const int steps = (a.kbytes + 127) / 128;
  int best = k64x128;
  double least = 0;
  for (int i = 0; i < kShapes; ++i) {
    const ShapeTime& t = times[i];
    if (t.tokens == 0) continue;
    const double tiles = live == 1 ? (a.rows + t.tokens - 1) / t.tokens
                                   : live * std::max(1.0, static_cast<double>(a.rows) / live / t.tokens + 0.5);
    const double blocks = tiles * std::ceil(n / t.channels);
    const double time =
        (steps + t.groups - 1) / t.groups * std::max<double>(t.latency, blocks / cus * t.cost);
    if (least == 0 || time < least) {
      least = time;
      best = i;
    }
  }
  return static_cast<Shape>(best);
}

template <typename T, bool kGated, int kOut>
hipError_t launch_typed(const GroupedArgs& a, int cus, hipStream_t s) {
  const Shape shape = choose_shape(a, cus);
  if constexpr (!std::is_same<T, F32Tag>::value) {
    if (shape == kWide) return launch_wide<T, kGated, kOut>(a, s);
    if (shape == k128x256) return launch_tile<T, kGated, kOut, 128, 256, 2, 4, 1, 3>(a, s);
  }
  switch (shape) {
    case k64x64: return launch_tile<T, kGated, kOut, 64, 64, 2, 2, 1, 4>(a, s);
    case k32x64: return launch_tile<T, kGated, kOut, 32, 64, 1, 2, 1, 4>(a, s);
    case k32x32by2: return launch_tile<T, kGated, kOut, 32, 32, 2, 1, 2, 4>(a, s);
    case k32x32by4: return launch_tile<T, kGated, kOut, 32, 32, 2, 1, 4, 3>(a, s);
    default: return launch_tile<T, kGated, kOut, 64, 128, 2, 4, 1, 3>(a, s);
  }
}

template <typename T>
hipError_t launch_type(const GroupedArgs& a, int cus, hipStream_t s) {
  if (a.out_dtype == PROX_F32)
    return a.w_gate ? launch_typed<T, true, PROX_F32>(a, cus, s) : launch_typed<T, false, PROX_F32>(a, cus, s);
  return a.w_gate ? launch_typed<T, true, PROX_BF16>(a, cus, s) : launch_typed<T, false, PROX_BF16>(a, cus, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, int cus, hipStream_t s) {
  if (a.wdtype == PROX_BF16) return launch_type<Bf16Tag>(a, cus, s);
  if (a.wdtype == PROX_F32) return launch_type<F32Tag>(a, cus, s);
  return launch_type<Fp8Tag>(a, cus, s);
}

}  // namespace prox
