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

typedef const __attribute__((address_space(1))) void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// 16 bytes per lane from memory to LDS at base + 16 * lane (base is uniform).
__device__ __forceinline__ void load_lds16(const void* src, void* base) {
  __builtin_amdgcn_global_load_lds((gptr_t)(src), (lptr_t)(base), 16, 0, 0);
}

struct Item {
  int group, row0, rows, channel_tile;  // rows: those of the tile, 1 .. BT
};

// The item-th (token tile, channel tile) of the launch.  Items run group by
// group; within a group the token tiles run fastest, so that neighbouring
// blocks share the group's weights.  False: there is no such item.
__device__ __forceinline__ bool find_item(const GroupedArgs& a, int bt, int channel_tiles, int item, Item* shared,
                                          int* wave_total) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  if (a.offsets == nullptr) {
    const int tiles = (a.rows + bt - 1) / bt;
    if (item >= tiles * channel_tiles) return false;
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
  if (item >= total * channel_tiles) return false;
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
__device__ __forceinline__ void store4(const GroupedArgs& a, int64_t row, int j, const float v[4]) {
  if constexpr (kOut == PROX_F32) {
    float* p = reinterpret_cast<float*>(a.out + row * a.out_stride) + j;
    if (a.vec_out && j + 4 <= a.n) {
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < a.n) p[i] = v[i];
    }
  } else {
    __bf16* p = reinterpret_cast<__bf16*>(a.out + row * a.out_stride) + j;
    if (a.vec_out && j + 4 <= a.n) {
      *reinterpret_cast<bf16x4_t*>(p) = bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < a.n) p[i] = (__bf16)v[i];
    }
  }
}

// One block: BT tokens x BC weight rows (gated: BC / 2 channels, up and gate in
// turn by sixteen rows), four waves of (BC / 2) x (BT / 2).
template <typename T, bool kGated, int kOut, int BT, int BC>
__global__ void __launch_bounds__(256) grouped_kernel(GroupedArgs a) {
  constexpr int kWaves = 4, FC = BC / 32, FT = BT / 32;  // fragments of 16 per wave
  constexpr bool kFp8 = std::is_same<T, Fp8Tag>::value;
  __shared__ __attribute__((aligned(16))) uint8_t sw[BC * 128];
  __shared__ __attribute__((aligned(16))) uint8_t sx[BT * 128];
  __shared__ Item s_item;
  __shared__ int s_total[kWaves];
  const int chan_per_tile = kGated ? BC / 2 : BC;
  const int channel_tiles = (a.n + chan_per_tile - 1) / chan_per_tile;
  if (!find_item(a, BT, channel_tiles, blockIdx.x, &s_item, s_total)) return;
  const Item it = s_item;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wc = wave >> 1, wt = wave & 1;  // this wave's channel half and token half
  const int c0 = it.channel_tile * chan_per_tile;

  // rows that this lane copies: eight rows per wave and copy, lane l the chunk
  // at place l % 8 of row l / 8
  const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
  const uint8_t* wsrc[BC / 8 / kWaves];
  const uint8_t* xsrc[BT / 8 / kWaves];
#pragma unroll
  for (int i = 0; i < BC / 8 / kWaves; ++i) {
    const int r = (i * kWaves + wave) * 8 + crow;
    const int j = kGated ? c0 + (r >> 5) * 16 + (r & 15) : c0 + r;
    const uint8_t* base = kGated && (r & 16) ? a.w_gate : a.w;
    wsrc[i] = j < a.n ? base + it.group * a.w_group + j * a.w_stride + chunk * 16 : nullptr;
  }
#pragma unroll
  for (int i = 0; i < BT / 8 / kWaves; ++i) {
    const int r = (i * kWaves + wave) * 8 + crow;
    int src = -1;
    if (r < it.rows) src = a.row_index ? a.row_index[it.row0 + r] : it.row0 + r;
    xsrc[i] = src >= 0 && src < a.a_rows ? a.a + src * a.a_stride + chunk * 16 : nullptr;
  }
  // fp8: the scale rows of this lane's tokens and of its channels
  const float* xs[FT];
  const float* wsc[FC];
  if constexpr (kFp8) {
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      const int r = (wt * FT + t) * 16 + (lane & 15);
      int src = -1;
      if (r < it.rows) src = a.row_index ? a.row_index[it.row0 + r] : it.row0 + r;
      xs[t] = src >= 0 && src < a.a_rows ? a.a_scale + static_cast<int64_t>(src) * a.kblocks : nullptr;
    }
#pragma unroll
    for (int f = 0; f < FC; ++f) {
      const int frag = wc * FC + f;
      const int j = min(a.n - 1, kGated ? c0 + (frag >> 1) * 16 : c0 + frag * 16);
      const float* base = kGated && (frag & 1) ? a.w_gate_scale : a.w_scale;
      wsc[f] = base + (static_cast<int64_t>(it.group) * a.nblocks + j / kScaleBlock) * a.kblocks;
    }
  }

  f32x4_t acc[FC][FT];
#pragma unroll
  for (int f = 0; f < FC; ++f)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[f][t] = f32x4_t{0, 0, 0, 0};

  for (int kb = 0; kb < a.kbytes; kb += 128) {
    const bool in = kb + chunk * 16 < a.kbytes;
#pragma unroll
    for (int i = 0; i < BC / 8 / kWaves; ++i)
      load_lds16(in && wsrc[i] ? static_cast<const void*>(wsrc[i] + kb) : &g_zero16, sw + (i * kWaves + wave) * 1024);
#pragma unroll
    for (int i = 0; i < BT / 8 / kWaves; ++i)
      load_lds16(in && xsrc[i] ? static_cast<const void*>(xsrc[i] + kb) : &g_zero16, sx + (i * kWaves + wave) * 1024);
    __syncthreads();
    Frag wf[FC], xf[FT];
    const int row = lane & 15, quad = lane >> 4;
#pragma unroll
    for (int f = 0; f < FC; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wf[f].c[h] = *reinterpret_cast<const u32x4_t*>(sw + ((wc * FC + f) * 16 + row) * 128 +
                                                       (((h * 4 + quad) ^ (row & 7)) << 4));
#pragma unroll
    for (int t = 0; t < FT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        xf[t].c[h] = *reinterpret_cast<const u32x4_t*>(sx + ((wt * FT + t) * 16 + row) * 128 +
                                                       (((h * 4 + quad) ^ (row & 7)) << 4));
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      float xscale = 0.f;
      if constexpr (kFp8) xscale = xs[t] ? xs[t][kb >> 7] : 0.f;
#pragma unroll
      for (int f = 0; f < FC; ++f) {
        if constexpr (kFp8) {
          const f32x4_t part = mma<T>(wf[f], xf[t], f32x4_t{0, 0, 0, 0});
          const float sc = xscale * wsc[f][kb >> 7];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(part[i], sc, acc[f][t][i]);
        } else {
          acc[f][t] = mma<T>(wf[f], xf[t], acc[f][t]);
        }
      }
    }
    __syncthreads();
  }

  const int quad = lane >> 4;
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    const int r = (wt * FT + t) * 16 + (lane & 15);
    if (r >= it.rows) continue;
#pragma unroll
    for (int f = 0; f < FC; f += kGated ? 2 : 1) {
      const int frag = wc * FC + f;
      const int j = (kGated ? c0 + (frag >> 1) * 16 : c0 + frag * 16) + quad * 4;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = kGated ? acc[f][t][i] * gate_act(acc[f + (kGated ? 1 : 0)][t][i], a.act) : acc[f][t][i];
      store4<kOut>(a, static_cast<int64_t>(it.row0) + r, j, v);
    }
  }
}

template <typename T, bool kGated, int kOut>
hipError_t launch_typed(const GroupedArgs& a, hipStream_t s) {
  constexpr int BT = 64, BC = 128;
  const int chan = kGated ? BC / 2 : BC;
  const int64_t tiles = a.rows / BT + std::min(a.n_groups, a.rows);
  const int64_t grid = tiles * ((a.n + chan - 1) / chan);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  grouped_kernel<T, kGated, kOut, BT, BC><<<dim3(static_cast<unsigned>(grid)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
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
