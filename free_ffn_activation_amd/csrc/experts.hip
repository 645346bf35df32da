// The operators around the products of a routed FFN: the router
// (prox_expert_route), the quantizer to e4m3 (prox_fp8_quantize) and the
// weighted sum of a token's expert rows (prox_expert_combine).
#include <float.h>

#include "experts_internal.h"
#include "prox_device.h"

namespace prox {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;

// ------------------------------------------------------------------- router
// A logit as an unsigned key: larger keys are larger logits, 0 (-inf) is never
// chosen, NaN comes first and makes the token's weights NaN; +inf counts as the
// largest finite value, so that the softmax below has no inf - inf.
__device__ __forceinline__ uint32_t route_key(float z) {
  if (z != z) return 0xFFFFFFFFu;
  if (z == -INFINITY) return 0u;
  const uint32_t b = __float_as_uint(fminf(z, FLT_MAX) + 0.0f);  // -0 orders with +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float route_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// op over the kLanes neighbouring lanes of a token, to every one of them: rotations
// inside a row of sixteen, then exchanges of rows and of halves of the wave.  (In
// every step both partners combine the same two values, so that fp32 sums agree.)
template <int kLanes, typename Op>
__device__ __forceinline__ uint32_t token_all(uint32_t v, Op op) {
#define PROX_ROTATE(n) \
  v = op(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + n, 0xF, 0xF, false)))
  PROX_ROTATE(8);
  PROX_ROTATE(4);
  PROX_ROTATE(2);
  PROX_ROTATE(1);
#undef PROX_ROTATE
  if constexpr (kLanes >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  if constexpr (kLanes == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(r[0], r[1]);
  }
  return v;
}

constexpr int kPlaceThreads = 1024;
constexpr int kRouteSub = 64;      // tokens of one bitmap pass: the bits of a word
constexpr int kRouteSmall = 32;    // tokens of a block of a small launch
constexpr int kRouteBlocks = 256;  // blocks at most
static_assert(kRouteSmall * kRouteBlocks < 1 << 16, "sums of byte counts are kept two to a word");

// Bytes of a block's counts where each is one byte.
__host__ __device__ inline int byte_counts(int experts) { return (experts + 3) / 4 * 4; }

// Threads of a block that chooses: for kRouteSmall tokens at once, if a block can.
__host__ __device__ constexpr int choose_threads(int lanes) {
  return lanes * kRouteSmall < 1024 ? lanes * kRouteSmall : 1024;
}

// Tokens per block: whole passes of kRouteSub beyond kRouteBlocks blocks of
// kRouteSmall.
__host__ __device__ inline int route_tokens_per_block(int tokens) {
  if (tokens <= kRouteSmall * kRouteBlocks) return kRouteSmall;
  const int per = (tokens + kRouteBlocks - 1) / kRouteBlocks;
  return (per + kRouteSub - 1) / kRouteSub * kRouteSub;
}

// The top_k of a token by kLanes lanes, 64 / kLanes tokens a wave: lane l of a token
// holds the experts l + kLanes i, i < kPer, and its slots l and l + kLanes.  Each round
// takes the token's largest key, then the lowest expert that has it, by token_all.  A
// round is a chain of dependent instructions, so what bounds a launch is their number
// per token (the logits of 8191 x 128 are read in 0.6 us, the launch takes 6; 65536 x
// 128 in fp32: 13,700 vector instructions a SIMD, of four cycles each, are some 26 of
// its 31 us): several tokens share one instruction (with the same second launch, us:
// 65536 tokens of 128 experts 39.6, a wave per token 73; 8191 of 512 23 and 56).  A whole
// wave finds the lowest expert by ballots, which are shorter than its second reduction
// (1024 experts: 77 and 82).  id: the experts of this lane's slots, or -1.
template <int kPer, int kLanes>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int end, int lane, int (&id)[2]) {
  constexpr int kSlots = kLanes < kMaxTopK ? 2 : 1;
  const auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
  const auto smaller = [](uint32_t x, uint32_t y) { return min(x, y); };
  const auto sum = [](uint32_t x, uint32_t y) { return __float_as_uint(__uint_as_float(x) + __uint_as_float(y)); };
  uint32_t key[kPer], my_key[2] = {0, 0};
  // lanes without a logit read another one, so that all loads are under way at once
  const size_t base = static_cast<size_t>(min(t, end - 1)) * a.experts;
  float z[kPer];
  if (a.logits_dtype == PROX_F32) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) z[i] = load_elem<F32Tag>(a.logits, base + min(lane + kLanes * i, a.experts - 1));
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) z[i] = load_elem<Bf16Tag>(a.logits, base + min(lane + kLanes * i, a.experts - 1));
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = t < end && lane + kLanes * i < a.experts ? route_key(z[i]) : 0;
  id[0] = id[1] = -1;
  float top = 0.f, rest = 0.f;  // rest: renormalize 0, the lane's share of the sum over all experts
  for (int s = 0; s < a.top_k; ++s) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, key[i]);
    best = token_all<kLanes>(best, larger);
    if (s == 0) {
      top = route_value(best);
      if (!a.renormalize) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (key[i] != 0) rest += expf(route_value(key[i]) - top);
          __builtin_amdgcn_sched_barrier(0);  // side by side they take all registers
        }
      }
    }
    uint32_t e = 0xFFFFFFFFu;
    if constexpr (kLanes == 64) {
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        const uint64_t has = __ballot(key[i] == best);
        if (has) e = 64 * i + __builtin_ctzll(has);
      }
    } else {
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i)
        if (key[i] == best) e = lane + kLanes * i;
      e = token_all<kLanes>(e, smaller);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e == static_cast<uint32_t>(lane + kLanes * i)) key[i] = 0;
#pragma unroll
    for (int h = 0; h < kSlots; ++h)
      if (best != 0 && lane + kLanes * h == s) {  // best 0: no expert is left
        my_key[h] = best;
        id[h] = static_cast<int>(e);
      }
  }
  float p[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) p[h] = id[h] >= 0 ? expf(route_value(my_key[h]) - top) : 0.f;
  const float total =
      __uint_as_float(token_all<kLanes>(__float_as_uint(a.renormalize ? p[0] + p[1] : rest), sum));
#pragma unroll
  for (int h = 0; h < kSlots; ++h)
    if (t < end && lane + kLanes * h < a.top_k) {
      const size_t o = static_cast<size_t>(t) * a.top_k + lane + kLanes * h;
      a.expert_idx[o] = id[h];
      a.weight[o] = id[h] >= 0 ? p[h] / total : 0.f;
    }
}

// Exclusive sums of count[0 .. experts) into start, by the whole block; returns
// the total.  Ends behind a barrier.
__device__ __forceinline__ int route_offsets(const int* count, int* start, int experts, int* wave_total) {
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int per = (experts + nthr - 1) / nthr;  // neighbouring experts of a thread
  int mine = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < experts) mine += count[tid * per + i];
  int at = wave_inclusive_scan_int(mine);
  if ((tid & 63) == 63) wave_total[tid >> 6] = at;
  __syncthreads();
  at -= mine;
  int rows = 0;
  for (int w = 0; w < nthr >> 6; ++w) {
    if (w < (tid >> 6)) at += wave_total[w];
    rows += wave_total[w];
  }
  for (int i = 0; i < per; ++i)
    if (tid * per + i < experts) {
      start[tid * per + i] = at;
      at += count[tid * per + i];
    }
  __syncthreads();
  return rows;
}

// Up to kTokens tokens, all in one block.  The chosen experts are kept as one bitmap
// word per expert (bit = token): a token takes an expert at most once, so its place
// among the expert's tokens is a population count.
template <int kPer, int kLanes, int kTokens>
__global__ void __launch_bounds__(1024) route_small_kernel(RouteArgs a) {
  typedef typename std::conditional<kTokens <= 32, uint32_t, unsigned long long>::type word_t;
  __shared__ word_t bits[kMaxExperts];
  __shared__ int count[kMaxExperts], start[kMaxExperts];
  __shared__ int wave_total[16];
  const int tid = threadIdx.x, lane = tid % kLanes;
  for (int e = tid; e < a.experts; e += 1024) bits[e] = 0;
  __syncthreads();
  constexpr int kAtOnce = 1024 / kLanes, kMine = (kTokens + kAtOnce - 1) / kAtOnce;  // tokens; of a wave's lanes
  int id[kMine][2];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int t = tid / kLanes + kAtOnce * i;
    id[i][0] = id[i][1] = -1;
    if (t - (tid & 63) / kLanes < a.tokens) route_token<kPer, kLanes>(a, t, a.tokens, lane, id[i]);  // by whole waves
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (id[i][h] >= 0) atomicOr(&bits[id[i][h]], word_t{1} << t);
  }
  __syncthreads();
  for (int e = tid; e < a.experts; e += 1024) count[e] = __popcll(bits[e]);
  __syncthreads();
  const int rows = route_offsets(count, start, a.experts, wave_total);
  for (int e = tid; e < a.experts; e += 1024) a.offsets[e] = start[e];
  if (tid == 0) a.offsets[a.experts] = rows;
#pragma unroll
  for (int i = 0; i < kMine; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = tid / kLanes + kAtOnce * i, s = lane + kLanes * h, e = id[i][h];
      if (t >= a.tokens || s >= a.top_k) continue;
      int row = -1;
      if (e >= 0) {
        row = start[e] + __popcll(bits[e] & ((word_t{1} << t) - 1));
        a.row_token[row] = t;
      }
      a.row_of[t * a.top_k + s] = row;
    }
  for (int r = rows + tid; r < a.tokens * a.top_k; r += 1024) a.row_token[r] = -1;
}

// More tokens, first launch: experts and weights of the block's tokens, and how
// many rows each expert gets from them.
template <int kPer, int kLanes>
__global__ void __launch_bounds__(choose_threads(kLanes)) route_choose_kernel(RouteArgs a) {
  constexpr int kThreads = choose_threads(kLanes);
  __shared__ int count[kMaxExperts];
  const int per = route_tokens_per_block(a.tokens);
  const int t0 = blockIdx.x * per, t1 = min(a.tokens, t0 + per);
  for (int e = threadIdx.x; e < a.experts; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int t = t0; t < t1; t += kThreads / kLanes) {
    int id[2];
    route_token<kPer, kLanes>(a, t + threadIdx.x / kLanes, t1, threadIdx.x % kLanes, id);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (id[h] >= 0) atomicAdd(&count[id[h]], 1);
  }
  __syncthreads();
  if (per == kRouteSmall) {
    const int bytes = byte_counts(a.experts);
    uint8_t* p = reinterpret_cast<uint8_t*>(a.block_count) + static_cast<size_t>(blockIdx.x) * bytes;
    for (int e = threadIdx.x; e < bytes; e += kThreads) p[e] = static_cast<uint8_t>(e < a.experts ? count[e] : 0);
  } else {
    int* p = a.block_count + static_cast<size_t>(blockIdx.x) * a.experts;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) p[e] = count[e];
  }
}

// Second launch: every block adds up the counts of all blocks (so that no block
// waits for another), then places its own rows.  What bounds it is a chain of
// latencies: its own experts are read first, and the counts by all threads side by
// side; in blocks of kRouteSmall tokens they are bytes, four to a load, whose sums
// (kRouteSmall * kRouteBlocks at most) are kept two to a word.  (8191 tokens of 128
// experts: 5.5 us; with counts of 32 bits, its experts read after them, 7.0.)
template <bool kBytes>
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(RouteArgs a, int blocks) {
  __shared__ uint32_t next[kMaxExperts];   // rows of earlier blocks, then the next row of each expert
  __shared__ uint32_t total[kMaxExperts];
  __shared__ int start[kMaxExperts];
  __shared__ unsigned long long bits[kMaxExperts];
  __shared__ int wave_total[kPlaceThreads / 64];
  constexpr int kMine = kRouteSub * kMaxTopK / kPlaceThreads;  // slots of a thread in a pass
  const int tid = threadIdx.x, me = blockIdx.x;
  const int tpb = route_tokens_per_block(a.tokens);
  const int t0 = me * tpb, t1 = min(a.tokens, t0 + tpb);
  int mine[kMine];  // their experts, or -1
  const auto read = [&](int s0) {
    const int slots = min(kRouteSub, t1 - s0) * a.top_k;
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int i = tid + u * kPlaceThreads;
      mine[u] = i < slots ? a.expert_idx[static_cast<size_t>(s0) * a.top_k + i] : -1;
    }
  };
  const auto mark = [&] {
#pragma unroll
    for (int u = 0; u < kMine; ++u)
      if (mine[u] >= 0) atomicOr(&bits[mine[u]], 1ull << ((tid + u * kPlaceThreads) / a.top_k));
  };
  read(t0);
  for (int e = tid; e < kMaxExperts; e += kPlaceThreads) {
    next[e] = total[e] = 0;
    bits[e] = 0;
  }
  __syncthreads();
  // columns: experts, or fours of them; `side` blocks' counts are read side by side
  const int columns = kBytes ? byte_counts(a.experts) / 4 : a.experts;
  const int side = kPlaceThreads / columns, column = tid % columns;
  if (tid < side * columns) {
    if constexpr (kBytes) {
      uint32_t before[2] = {0, 0}, sum[2] = {0, 0};  // experts 0 and 2, 1 and 3 of the four
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.block_count) + column;
#pragma unroll 8
      for (int b = tid / columns; b < blocks; b += side) {
        const uint32_t c = p[static_cast<size_t>(b) * columns];
        const uint32_t c0 = c & 0x00FF00FFu, c1 = c >> 8 & 0x00FF00FFu;
        sum[0] += c0;
        sum[1] += c1;
        before[0] += b < me ? c0 : 0;
        before[1] += b < me ? c1 : 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        atomicAdd(&next[2 * column + h], before[h]);
        atomicAdd(&total[2 * column + h], sum[h]);
      }
    } else {
      uint32_t before = 0, sum = 0;
      const int* p = a.block_count + column;
#pragma unroll 16
      for (int b = tid / columns; b < blocks; b += side) {
        const uint32_t c = p[static_cast<size_t>(b) * columns];
        before += b < me ? c : 0;
        sum += c;
      }
      atomicAdd(&next[column], before);
      atomicAdd(&total[column], sum);
    }
  }
  mark();
  __syncthreads();
  if constexpr (kBytes) {  // to a word per expert
    uint32_t n = 0, m = 0;
    const int word = tid / 4 * 2 + (tid & 1), shift = (tid & 2) * 8;
    if (tid < a.experts) {
      n = next[word] >> shift & 0xFFFFu;
      m = total[word] >> shift & 0xFFFFu;
    }
    __syncthreads();
    if (tid < a.experts) {
      next[tid] = n;
      total[tid] = m;
    }
    __syncthreads();
  }
  const int rows = route_offsets(reinterpret_cast<const int*>(total), start, a.experts, wave_total);
  for (int e = tid; e < a.experts; e += kPlaceThreads) {
    if (me == 0) a.offsets[e] = start[e];
    next[e] += start[e];
  }
  if (me == 0 && tid == 0) a.offsets[a.experts] = rows;
  __syncthreads();
  for (int s0 = t0; s0 < t1; s0 += kRouteSub) {
    if (s0 > t0) {
      read(s0);
      __syncthreads();
      for (int e = tid; e < a.experts; e += kPlaceThreads) {
        next[e] += __popcll(bits[e]);
        bits[e] = 0;
      }
      __syncthreads();
      mark();
      __syncthreads();
    }
    const int slots = min(kRouteSub, t1 - s0) * a.top_k;
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int i = tid + u * kPlaceThreads;
      if (i >= slots) continue;
      const int t = i / a.top_k, e = mine[u];
      int row = -1;
      if (e >= 0) {
        row = static_cast<int>(next[e]) + __popcll(bits[e] & ((1ull << t) - 1));
        a.row_token[row] = s0 + t;
      }
      a.row_of[static_cast<size_t>(s0) * a.top_k + i] = row;
    }
  }
  // rows behind the last expert's
  const int all = a.tokens * a.top_k;
  for (int r = rows + me * kPlaceThreads + tid; r < all; r += blocks * kPlaceThreads) a.row_token[r] = -1;
}

// ---------------------------------------------------------------- quantizer
// 8 neighbouring values as fp32
template <typename T> __device__ __forceinline__ void load8(const uint8_t* p, float v[8]);
template <> __device__ __forceinline__ void load8<Bf16Tag>(const uint8_t* p, float v[8]) {
  const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(w[i]);
    v[2 * i + 1] = bf16hi(w[i]);
  }
}
template <> __device__ __forceinline__ void load8<F32Tag>(const uint8_t* p, float v[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x4_t w = reinterpret_cast<const f32x4_t*>(p)[h];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * h + i] = w[i];
  }
}

// The largest |v| as bits: integer order puts finite values below infinity and
// infinity below NaN, so a block with either is seen.
__device__ __forceinline__ uint32_t abs_bits8(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// The scale fp32(amax / 448); NaN where the block holds an infinity or NaN.
__device__ __forceinline__ float block_scale(uint32_t amax) {
  return amax < 0x7F800000u ? __uint_as_float(amax) / 448.0f : __uint_as_float(0x7FC00000u);
}

// fp32(v / scale) of N values, correctly rounded.  One division for the block:
// inv = fp32(1 / scale); each quotient then is v inv, corrected twice by its exact
// remainder.  The first correction leaves it within one step of the quotient, and
// from there, with a correctly rounded inv, the second gives the correctly rounded
// one (Markstein's theorem on division by fused multiply-add): 5 operations
// against the 10 and more of a division, 20 against 26 us for 8192 x 4096 values.
// Remainders must not underflow: below 2^-80 (a block of values that small) plain
// divisions.  Quotients so small that theirs do are codes of 0 either way.
// A scale of a few subnormal steps is rounded down by up to a third, so that
// quotients reach 672: they are held at the largest code, 448, since the conversion
// makes NaN of anything above 464.  Scales of 2^-136 and more are off by 2^-14 at
// most, and their quotients round to 448 by themselves.
template <int N>
__device__ __forceinline__ void divide(const float (&v)[N], float scale, float (&q)[N]) {
  if (scale < 0x1p-80f) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = scale == 0.f ? 0.f : fminf(fmaxf(v[i] / scale, -448.f), 448.f);
    return;
  }
  const float inv = 1.0f / scale;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = v[i] * inv;
    t = fmaf(fmaf(-t, scale, v[i]), inv, t);
    q[i] = fmaf(fmaf(-t, scale, v[i]), inv, t);
  }
}

// e4m3(fp32(v / scale)), four values a word.  Scale 0 (an all-zero block): zeros;
// scale NaN: NaN.
template <int N>
__device__ __forceinline__ void to_e4m3(const float (&v)[N], float scale, uint32_t (&r)[N / 4]) {
  float q[N];
  divide(v, scale, q);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
    r[i] = scale != scale ? 0x7F7F7F7Fu : static_cast<uint32_t>(w);
  }
}

// Rows: eight lanes hold the 128 values of a block, sixteen each.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantizeArgs a, int kblocks) {
  const int64_t block = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;
  if (block >= static_cast<int64_t>(a.rows) * kblocks) return;
  // kblocks divides without a 64-bit division where the block number fits 32 bits
  const int64_t row = block <= 0xFFFFFFFFll ? static_cast<uint32_t>(block) / static_cast<uint32_t>(kblocks)
                                            : block / kblocks;
  const int col = static_cast<int>(block - row * kblocks) * kScaleBlock + (threadIdx.x & 7) * 16;
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  const bool in = col < a.k;  // k is a multiple of 16
  if (in) {
    const uint8_t* p = a.x + row * a.x_stride + static_cast<int64_t>(col) * sizeof(typename T::storage);
    load8<T>(p, *reinterpret_cast<float(*)[8]>(v));
    load8<T>(p + 8 * sizeof(typename T::storage), *reinterpret_cast<float(*)[8]>(v + 8));
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  const float scale = block_scale(m);
  uint32_t r[4];
  to_e4m3(v, scale, r);
  if (in) *reinterpret_cast<u32x4_t*>(a.q + row * a.q_stride + col) = u32x4_t{r[0], r[1], r[2], r[3]};
  if ((threadIdx.x & 7) == 0) a.scale[block] = scale;
}

// Square blocks of weights: one workgroup per 128 x 128.
template <typename T>
__global__ void __launch_bounds__(256) quantize_square_kernel(QuantizeArgs a) {
  __shared__ uint32_t wave_max[4];
  const int kblocks = (a.k + kScaleBlock - 1) / kScaleBlock;
  const int64_t rb = blockIdx.x / kblocks;
  const int cb = blockIdx.x % kblocks;
  const int col = cb * kScaleBlock + (threadIdx.x & 15) * 8;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = rb * kScaleBlock + i * 16 + (threadIdx.x >> 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (row < a.rows && col < a.k)
      load8<T>(a.x + row * a.x_stride + static_cast<int64_t>(col) * sizeof(typename T::storage), v[i]);
    m = max(m, abs_bits8(v[i]));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
  const float scale = block_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = rb * kScaleBlock + i * 16 + (threadIdx.x >> 4);
    uint32_t r[2];
    to_e4m3(v[i], scale, r);
    if (row < a.rows && col < a.k) *reinterpret_cast<uint2*>(a.q + row * a.q_stride + col) = uint2{r[0], r[1]};
  }
  if (threadIdx.x == 0) a.scale[rb * kblocks + cb] = scale;
}

// ------------------------------------------------------------------ combine
// A thread adds up kVec neighbouring values of one token, slot by slot in
// fp32; the order of the sum is that of the slots, whatever the launch.
template <typename T, int kOut, int kVec>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a, int blocks_per_token) {
  const int token = blockIdx.x / blocks_per_token;
  const int j = ((blockIdx.x % blocks_per_token) * blockDim.x + threadIdx.x) * kVec;
  if (j >= a.n) return;
  float acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
  const size_t slot0 = static_cast<size_t>(token) * a.top_k;
  // four slots' rows are read side by side; a slot without a row adds nothing
  for (int s0 = 0; s0 < a.top_k; s0 += 4) {
    float v[4][kVec], w[4];
    bool use[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = min(s0 + u, a.top_k - 1);
      const int row = a.row_of[slot0 + s];
      use[u] = s0 + u < a.top_k && row >= 0 && row < a.h_rows;
      w[u] = a.weight[slot0 + s];
      if (use[u]) {
        const uint8_t* p = a.h + row * a.h_stride;
        if constexpr (kVec == 8) load8<T>(p + static_cast<int64_t>(j) * sizeof(typename T::storage), v[u]);
        else v[u][0] = load_elem<T>(p, j);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (use[u]) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i] = fmaf(w[u], v[u][i], acc[i]);
      }
  }
  uint8_t* q = a.y + token * a.y_stride;
  if constexpr (kOut == PROX_F32) {
    float* y = reinterpret_cast<float*>(q) + j;
    if constexpr (kVec == 8) {
      reinterpret_cast<f32x4_t*>(y)[0] = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
      reinterpret_cast<f32x4_t*>(y)[1] = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
    } else {
      y[0] = acc[0];
    }
  } else {
    __bf16* y = reinterpret_cast<__bf16*>(q) + j;
    if constexpr (kVec == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        reinterpret_cast<bf16x4_t*>(y)[h] = bf16x4_t{(__bf16)acc[4 * h], (__bf16)acc[4 * h + 1],
                                                     (__bf16)acc[4 * h + 2], (__bf16)acc[4 * h + 3]};
    } else {
      y[0] = (__bf16)acc[0];
    }
  }
}

// kVec 8 needs whole vectors in aligned rows; other n, strides and addresses take
// kVec 1, each element a load of its own.
template <typename T, int kOut, int kVec>
hipError_t launch_combine_typed(const CombineArgs& a, hipStream_t s) {
  const int threads = std::min(256, ((a.n + kVec - 1) / kVec + 63) / 64 * 64);
  const int per = (a.n + kVec * threads - 1) / (kVec * threads);
  const int64_t grid = static_cast<int64_t>(a.tokens) * per;
  if (!grid_fits(grid, threads)) return hipErrorInvalidConfiguration;
  combine_kernel<T, kOut, kVec><<<dim3(static_cast<unsigned>(grid)), dim3(threads), 0, s>>>(a, per);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_combine_type(const CombineArgs& a, hipStream_t s) {
  if (a.y_dtype == PROX_F32)
    return a.vec ? launch_combine_typed<T, PROX_F32, 8>(a, s) : launch_combine_typed<T, PROX_F32, 1>(a, s);
  return a.vec ? launch_combine_typed<T, PROX_BF16, 8>(a, s) : launch_combine_typed<T, PROX_BF16, 1>(a, s);
}

int route_blocks(int tokens) {
  const int per = route_tokens_per_block(tokens);
  return std::max(1, (tokens + per - 1) / per);
}

}  // namespace

size_t route_workspace(int tokens, int experts) {
  return (static_cast<size_t>(route_blocks(tokens)) * experts * sizeof(int) + 255) & ~static_cast<size_t>(255);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const auto launch = [&](auto kernel, int blocks, int threads) {
    kernel<<<dim3(blocks), dim3(threads), 0, s>>>(a);
    return hipGetLastError();
  };
  const auto launch_small = [&](auto kernel) { return launch(kernel, 1, 1024); };
  // One block, with as many lanes per token as it has: fewer keys a lane, shorter
  // rounds.  (us: 1 token of 64 experts 3.5, 64 tokens 5.6, 65 by the two launches 7.5; 64
  // tokens of 512 experts would take 17.5 in one block, by the two launches 13.6.)
  if (a.tokens <= 16) {
    if (a.experts <= 64) return launch_small(route_small_kernel<1, 64, 16>);
    if (a.experts <= 128) return launch_small(route_small_kernel<2, 64, 16>);
    if (a.experts <= 256) return launch_small(route_small_kernel<4, 64, 16>);
    if (a.experts <= 512) return launch_small(route_small_kernel<8, 64, 16>);
    return launch_small(route_small_kernel<16, 64, 16>);
  }
  if (a.tokens <= 64 && a.experts <= 128)
    return a.experts <= 64 ? launch_small(route_small_kernel<4, 16, 64>) : launch_small(route_small_kernel<8, 16, 64>);
  if (a.tokens <= 32) {
    if (a.experts <= 256) return launch_small(route_small_kernel<8, 32, 32>);
    if (a.experts <= 512) return launch_small(route_small_kernel<16, 32, 32>);
    return launch_small(route_small_kernel<16, 64, 32>);
  }
  // Two launches; a block has all its tokens at once where it can.  (us, tokens x
  // experts, keys by lanes per token: 65536 x 64: 4 x 16 25.6, 2 x 32 29.0; 65536 x 128:
  // 4 x 32 39.6, 8 x 16 50.9; 16384 x 256: 8 x 32 21.5, 4 x 64 26.9; 65536 x 512: 16 x 32
  // 81, 8 x 64 100; 8191 x 1024: 16 x 64 41.5, 32 x 32 43.0)
  const int blocks = route_blocks(a.tokens);
  const hipError_t e = a.experts <= 64    ? launch(route_choose_kernel<4, 16>, blocks, choose_threads(16))
                       : a.experts <= 128 ? launch(route_choose_kernel<4, 32>, blocks, choose_threads(32))
                       : a.experts <= 256 ? launch(route_choose_kernel<8, 32>, blocks, choose_threads(32))
                       : a.experts <= 512 ? launch(route_choose_kernel<16, 32>, blocks, choose_threads(32))
                                          : launch(route_choose_kernel<16, 64>, blocks, choose_threads(64));
  if (e != hipSuccess) return e;
  if (route_tokens_per_block(a.tokens) == kRouteSmall)
    route_place_kernel<true><<<dim3(blocks), dim3(kPlaceThreads), 0, s>>>(a, blocks);
  else
    route_place_kernel<false><<<dim3(blocks), dim3(kPlaceThreads), 0, s>>>(a, blocks);
  return hipGetLastError();
}

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  const int64_t kblocks = (a.k + kScaleBlock - 1) / kScaleBlock;
  const int64_t grid = a.block_rows == 1 ? (a.rows * kblocks + 31) / 32
                                         : (a.rows + kScaleBlock - 1) / kScaleBlock * kblocks;
  if (!grid_fits(grid, 256)) return hipErrorInvalidConfiguration;
  const dim3 g(static_cast<unsigned>(grid)), b(256);
  if (a.block_rows == 1) {
    if (a.x_dtype == PROX_F32) quantize_rows_kernel<F32Tag><<<g, b, 0, s>>>(a, static_cast<int>(kblocks));
    else quantize_rows_kernel<Bf16Tag><<<g, b, 0, s>>>(a, static_cast<int>(kblocks));
  } else {
    if (a.x_dtype == PROX_F32) quantize_square_kernel<F32Tag><<<g, b, 0, s>>>(a);
    else quantize_square_kernel<Bf16Tag><<<g, b, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s) {
  return a.h_dtype == PROX_F32 ? launch_combine_type<F32Tag>(a, s) : launch_combine_type<Bf16Tag>(a, s);
}

}  // namespace prox
