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
// The matrix cores add eight neighbouring products at the exponent of the
// largest and cut each off at 2^-13 of it (measured, both e4m3 instructions
// alike); eights, and the fp32 sum of the 128-blocks, are added exactly.  That
// is far below the codes' own 2^-4, and twice as fast as bf16 products of the
// widened codes, so it is taken as it is.
template <>
__device__ __forceinline__ f32x4_t mma<Fp8Tag>(const Frag& w, const Frag& x, f32x4_t acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8_t, w),
                                                          __builtin_bit_cast(i32x8_t, x), acc, 0, 0, 0, 0, 0, 0);
}

// Sixteen zero bytes: the source of rows and chunks that do not exist.
__device__ const u32x4_t g_zero16 = {0, 0, 0, 0};

typedef __attribute__((address_space(3))) uint8_t* lds_ptr_t;
__device__ __forceinline__ uint32_t lds_offset(void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr_t)(p)));
}

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

struct Item {
  int group, row0, rows, channel_tile;  // rows: those of the tile, 1 .. BT
};

// The (token tile, channel tile) of this block.  Items run group by group;
// within a group the token tiles run fastest.  Blocks go round the eight XCDs,
// each with an L2 of its own: XCD x takes the x-th eighth of the items, so that
// the blocks that share a group's weights share an L2.  False: no item is left.
__device__ __forceinline__ bool find_item(const GroupedArgs& a, int bt, int channel_tiles, Item* shared,
                                          int* wave_total) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int xcd = blockIdx.x & 7, nth = blockIdx.x >> 3;
  if (a.offsets == nullptr) {
    const int tiles = (a.rows + bt - 1) / bt, items = tiles * channel_tiles;
    const int share = (items + 7) >> 3, item = xcd * share + nth;
    if (nth >= share || item >= items) return false;
    if (tid == 0) {
      const int m = item % tiles;
      *shared = {0, m * bt, min(bt, a.rows - m * bt), item / tiles};
    }
    __syncthreads();
    return true;
  }
  const int per = (a.n_groups + nthr - 1) / nthr;
  const int g0 = tid * per;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int g = g0 + i;
    if (g < a.n_groups) {
      const int lo = min(max(a.offsets[g], 0), a.rows), hi = min(max(a.offsets[g + 1], lo), a.rows);
      mine += (hi - lo + bt - 1) / bt;
    }
  }
  int before = wave_inclusive_scan_int(mine);
  if ((tid & 63) == 63) wave_total[tid >> 6] = before;
  __syncthreads();
  int total = 0;
  before -= mine;
  for (int w = 0; w < nthr >> 6; ++w) {
    if (w < (tid >> 6)) before += wave_total[w];
    total += wave_total[w];
  }
  const int items = total * channel_tiles;
  const int share = (items + 7) >> 3, item = xcd * share + nth;
  if (nth >= share || item >= items) return false;
  if (item >= before * channel_tiles && item < (before + mine) * channel_tiles) {
    for (int i = 0; i < per; ++i) {
      const int g = g0 + i;
      if (g >= a.n_groups) break;
      const int lo = min(max(a.offsets[g], 0), a.rows), hi = min(max(a.offsets[g + 1], lo), a.rows);
      const int tiles = (hi - lo + bt - 1) / bt;
      const int rem = item - before * channel_tiles;
      if (rem < tiles * channel_tiles) {
        const int m = rem % tiles;
        *shared = {g, lo + m * bt, min(bt, hi - lo - m * bt), rem / tiles};
        break;
      }
      before += tiles;
    }
  }
  __syncthreads();
  return true;
}

template <int kOut>
__device__ __forceinline__ void store4(const GroupedArgs& a, bool whole, int64_t row, int j, const float v[4]) {
  if constexpr (kOut == PROX_F32) {
    float* p = reinterpret_cast<float*>(a.out + row * a.out_stride) + j;
    if (whole) {
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < a.n) p[i] = v[i];
    }
  } else {
    __bf16* p = reinterpret_cast<__bf16*>(a.out + row * a.out_stride) + j;
    if (whole) {
      *reinterpret_cast<bf16x4_t*>(p) = bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < a.n) p[i] = (__bf16)v[i];
    }
  }
}

// Waits until at most kLeft of this wave's memory-to-LDS copies are under way,
// and for its LDS reads, then for the other waves of the block.
template <int kLeft>
__device__ __forceinline__ void wait_copies_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

// One block: BT tokens x BC weight rows (gated: BC / 2 channels, up and gate in
// turn by sixteen rows), WC x WT waves.  Two LDS buffers: while the waves
// multiply step s, the copies of step s + 1 are under way.
template <typename T, bool kGated, int kOut, int BT, int BC, int WT, int WC>
__global__ void __launch_bounds__(64 * WT * WC) grouped_kernel(GroupedArgs a) {
  constexpr int kWaves = WT * WC, FC = BC / 16 / WC, FT = BT / 16 / WT;  // fragments of 16 per wave
  constexpr int NW = BC / 8 / kWaves, NX = BT / 8 / kWaves;              // copies per wave and step
  constexpr bool kFp8 = std::is_same<T, Fp8Tag>::value;
  static_assert(NW * 8 * kWaves == BC && NX * 8 * kWaves == BT && FC * 16 * WC == BC && FT * 16 * WT == BT, "tile");
  static_assert(FC <= 8 && 128 % (FC * 16) == 0, "a wave's channels lie in one scale block");
  static_assert(!kGated || FC % 2 == 0, "up and gate of a channel belong to one wave");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * (BC + BT) * 128];
  __shared__ Item s_item;
  __shared__ int s_total[kWaves];
  const int chan_per_tile = kGated ? BC / 2 : BC;
  const int channel_tiles = (a.n + chan_per_tile - 1) / chan_per_tile;
  if (!find_item(a, BT, channel_tiles, &s_item, s_total)) return;
  const Item it = {__builtin_amdgcn_readfirstlane(s_item.group), __builtin_amdgcn_readfirstlane(s_item.row0),
                   __builtin_amdgcn_readfirstlane(s_item.rows), __builtin_amdgcn_readfirstlane(s_item.channel_tile)};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave / WT, wt = wave % WT;  // this wave's share of the channels and of the tokens
  const int c0 = it.channel_tile * chan_per_tile;

  // Rows that this lane copies: eight rows per wave and copy, lane l the chunk
  // at place l % 8 of row l / 8.  Rows past the last token or channel of the
  // tile repeat a row that exists; their results are not stored.
  const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
  // uniform: the tile's first channel, up and gate
  const int64_t first = it.group * a.w_group + c0 * a.w_stride;
  const uint8_t* const w_up = a.w + first;
  const uint8_t* const w_gate = kGated ? a.w_gate + first : w_up;
  uint32_t woff[NW];  // below 2^31: at most 256 rows of less than 2^23 bytes
  const uint8_t* xsrc[NX];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int r = (i * kWaves + wave) * 8 + crow;
    const int j = min(kGated ? (r >> 5) * 16 + (r & 15) : r, a.n - 1 - c0);
    woff[i] = static_cast<uint32_t>(j) * static_cast<uint32_t>(a.w_stride) + chunk * 16;
  }
  const auto source = [&](int r) {  // the row of a for row r of the tile, or -1
    r = it.row0 + min(r, it.rows - 1);
    const int src = a.row_index ? a.row_index[r] : r;
    return src < a.a_rows ? src : -1;
  };
#pragma unroll
  for (int i = 0; i < NX; ++i)
    xsrc[i] = a.a + max(source((i * kWaves + wave) * 8 + crow), 0) * a.a_stride + chunk * 16;
  // fp8: the scales of this lane's tokens and of this wave's channels, which
  // lie in one block of 128 (up and gate each)
  const float* xs[FT];
  const float *wsc_up = nullptr, *wsc_gate = nullptr;
  if constexpr (kFp8) {
#pragma unroll
    for (int t = 0; t < FT; ++t)
      xs[t] = a.a_scale + static_cast<int64_t>(max(source((wt * FT + t) * 16 + (lane & 15)), 0)) * a.kblocks;
    const int j = min(c0 + wc * FC * (kGated ? 8 : 16), a.n - 1);
    const int64_t block = (static_cast<int64_t>(it.group) * a.nblocks + j / kScaleBlock) * a.kblocks;
    wsc_up = a.w_scale + block;
    wsc_gate = kGated ? a.w_gate_scale + block : wsc_up;
  }

  f32x4_t acc[FC][FT];
#pragma unroll
  for (int f = 0; f < FC; ++f)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[f][t] = f32x4_t{0, 0, 0, 0};

  constexpr uint32_t kBuffer = (BC + BT) * 128;
  const uint32_t lds0 = lds_offset(lds);
  const auto copy = [&](int kb, uint32_t to) {
    to += lds0 + wave * 1024;
    if (kb + 128 <= a.kbytes) {
#pragma unroll
      for (int i = 0; i < NW; ++i)  // copy i holds up (even sixteens) or gate rows
        copy16((kGated && (((i * kWaves + wave) >> 1) & 1) ? w_gate : w_up) + kb, woff[i], to + i * (kWaves * 1024));
#pragma unroll
      for (int i = 0; i < NX; ++i) copy16(xsrc[i] + kb, to + BC * 128 + i * (kWaves * 1024));
    } else {  // the last step of a k that is no multiple of 128 bytes
      const bool in = kb + chunk * 16 < a.kbytes;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint8_t* w = (kGated && (((i * kWaves + wave) >> 1) & 1) ? w_gate : w_up) + kb + woff[i];
        copy16(in ? static_cast<const void*>(w) : &g_zero16, to + i * (kWaves * 1024));
      }
#pragma unroll
      for (int i = 0; i < NX; ++i)
        copy16(in ? static_cast<const void*>(xsrc[i] + kb) : &g_zero16, to + BC * 128 + i * (kWaves * 1024));
    }
  };
  const int row = lane & 15, quad = lane >> 4;
  const int place0 = ((quad) ^ (row & 7)) << 4, place1 = ((4 + quad) ^ (row & 7)) << 4;
  const auto multiply = [&](int kb, const uint8_t* from) {
    const uint8_t* pw = from + (wc * FC * 16 + row) * 128;
    const uint8_t* px = from + BC * 128 + (wt * FT * 16 + row) * 128;
    Frag xf[FT], wf[2];
    float xscale[FT], ws_up = 0.f, ws_gate = 0.f;
    if constexpr (kFp8) {
#pragma unroll
      for (int t = 0; t < FT; ++t) xscale[t] = xs[t][kb >> 7];
      ws_up = wsc_up[kb >> 7];
      ws_gate = kGated ? wsc_gate[kb >> 7] : ws_up;
    }
    wf[0].c[0] = *reinterpret_cast<const u32x4_t*>(pw + place0);
    wf[0].c[1] = *reinterpret_cast<const u32x4_t*>(pw + place1);
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      xf[t].c[0] = *reinterpret_cast<const u32x4_t*>(px + t * 2048 + place0);
      xf[t].c[1] = *reinterpret_cast<const u32x4_t*>(px + t * 2048 + place1);
    }
#pragma unroll
    for (int f = 0; f < FC; ++f) {
      // the next channels' fragment is read while this one is multiplied
      if (f + 1 < FC) {
        wf[(f + 1) & 1].c[0] = *reinterpret_cast<const u32x4_t*>(pw + (f + 1) * 2048 + place0);
        wf[(f + 1) & 1].c[1] = *reinterpret_cast<const u32x4_t*>(pw + (f + 1) * 2048 + place1);
      }
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        if constexpr (kFp8) {
          const f32x4_t part = mma<T>(wf[f & 1], xf[t], f32x4_t{0, 0, 0, 0});
          const float sc = xscale[t] * (kGated && (f & 1) ? ws_gate : ws_up);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(part[i], sc, acc[f][t][i]);
        } else {
          acc[f][t] = mma<T>(wf[f & 1], xf[t], acc[f][t]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  copy(0, 0);
  uint32_t now = 0;
  for (int kb = 0; kb < a.kbytes; kb += 128) {
    wait_copies_and_meet<0>();
    if (kb + 128 < a.kbytes) copy(kb + 128, now ^ kBuffer);
    multiply(kb, lds + now);
    now ^= kBuffer;
  }

  const auto result = [&](int f, int t, float v[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = kGated ? acc[f][t][i] * gate_act(acc[f + (kGated ? 1 : 0)][t][i], a.act) : acc[f][t][i];
  };
  const bool whole = a.vec_out && c0 + chan_per_tile <= a.n;  // uniform
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    const int r = (wt * FT + t) * 16 + (lane & 15);
    if (r >= it.rows) continue;
    const bool none = source(r) < 0;  // a row index outside a: zeros
#pragma unroll
    for (int f = 0; f < FC; f += kGated ? 2 : 1) {
      const int frag = wc * FC + f;
      const int j = (kGated ? c0 + (frag >> 1) * 16 : c0 + frag * 16) + quad * 4;
      float v[4];
      result(f, t, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = none ? 0.f : v[i];
      store4<kOut>(a, whole, static_cast<int64_t>(it.row0) + r, j, v);
    }
  }
}

template <typename T, bool kGated, int kOut, int BT, int BC, int WT, int WC>
hipError_t launch_tile(const GroupedArgs& a, hipStream_t s) {
  const int chan = kGated ? BC / 2 : BC;
  const int64_t tiles = a.rows / BT + std::min(a.n_groups, a.rows);
  const int64_t grid = (tiles * ((a.n + chan - 1) / chan) + 7) / 8 * 8;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  grouped_kernel<T, kGated, kOut, BT, BC, WT, WC><<<dim3(static_cast<unsigned>(grid)), dim3(64 * WT * WC), 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, bool kGated, int kOut>
hipError_t launch_typed(const GroupedArgs& a, hipStream_t s) {
  if (a.rows / a.n_groups >= 128) return launch_tile<T, kGated, kOut, 256, 256, 4, 2>(a, s);
  return launch_tile<T, kGated, kOut, 64, 128, 2, 2>(a, s);
}

template <typename T>
hipError_t launch_type(const GroupedArgs& a, hipStream_t s) {
  if (a.out_dtype == PROX_F32)
    return a.w_gate ? launch_typed<T, true, PROX_F32>(a, s) : launch_typed<T, false, PROX_F32>(a, s);
  return a.w_gate ? launch_typed<T, true, PROX_BF16>(a, s) : launch_typed<T, false, PROX_BF16>(a, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, int cus, hipStream_t s) {
  (void)cus;
  if (a.wdtype == PROX_BF16) return launch_type<Bf16Tag>(a, s);
  if (a.wdtype == PROX_F32) return launch_type<F32Tag>(a, s);
  return launch_type<Fp8Tag>(a, s);
}

}  // namespace prox
