// Host side of the routed-FFN entry points of include/prox.h: argument
// validation and launches.
#include <algorithm>

#include "experts_internal.h"

#define PROX_API extern "C" __attribute__((visibility("default")))

namespace prox {
namespace {

constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int kMaxDim = 1 << 24;                  // n and k
constexpr int64_t kMaxStride = int64_t{1} << 40;  // elements; keeps the sizes in bytes inside 64 bits
constexpr int64_t kMaxWeightRow = 1 << 23;        // bytes: the products' offsets inside a tile have 32 bits

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
int elem(int dtype) { return dtype == PROX_F32 ? 4 : dtype == PROX_BF16 ? 2 : 1; }
bool stride_fits(int64_t s) { return s >= -kMaxStride && s <= kMaxStride; }
int blocks128(int v) { return (v + kScaleBlock - 1) / kScaleBlock; }

prox_status check_experts(const prox_experts* e) {
  if (!e) return fail(PROX_ERR_INVALID_ARG, "experts descriptor is NULL");
  if (e->wdtype != PROX_F32 && e->wdtype != PROX_BF16 && e->wdtype != PROX_FP8)
    return fail(PROX_ERR_INVALID_ARG, "experts wdtype %d is none of PROX_F32, PROX_BF16, PROX_FP8", e->wdtype);
  if (e->reserved != 0) return fail(PROX_ERR_INVALID_ARG, "experts reserved must be 0");
  if (e->activation != PROX_ACT_SILU && e->activation != PROX_ACT_GELU_TANH)
    return fail(PROX_ERR_INVALID_ARG, "experts activation %d is neither PROX_ACT_SILU nor PROX_ACT_GELU_TANH",
                e->activation);
  if (e->n_groups < 1 || e->n < 1 || e->k < 1)
    return fail(PROX_ERR_INVALID_ARG, "experts n_groups %d, n %d and k %d must be positive", e->n_groups, e->n, e->k);
  if (e->n_groups > kMaxExperts || e->n > kMaxDim || e->k > kMaxDim)
    return fail(PROX_ERR_UNSUPPORTED, "experts n_groups %d above %d, or n %d or k %d above 2^24", e->n_groups,
                kMaxExperts, e->n, e->k);
  if (!stride_fits(e->row_stride) || !stride_fits(e->group_stride))
    return fail(PROX_ERR_UNSUPPORTED, "experts strides must be at most 2^40 elements");
  const int es = elem(e->wdtype);
  if (static_cast<int64_t>(e->k) * es % 16 != 0 || e->row_stride * es % 16 != 0 || e->group_stride * es % 16 != 0)
    return fail(PROX_ERR_UNSUPPORTED, "experts k and strides must be multiples of 16 bytes");
  if (e->row_stride * es >= kMaxWeightRow)
    return fail(PROX_ERR_UNSUPPORTED, "experts row_stride must be below 8 MiB");
  if (e->row_stride < e->k || e->group_stride < 0)
    return fail(PROX_ERR_INVALID_ARG, "experts row_stride is below k or group_stride is negative");
  if (!e->w || !aligned(e->w, 16) || !aligned(e->w_gate, 16))
    return fail(PROX_ERR_INVALID_ARG, "experts weights must be non-NULL and 16-byte aligned");
  if (e->wdtype == PROX_FP8) {
    if (!e->w_scale || (e->w_gate && !e->w_gate_scale))
      return fail(PROX_ERR_INVALID_ARG, "experts scales must be non-NULL for PROX_FP8");
    if (!aligned(e->w_scale, 4) || !aligned(e->w_gate_scale, 4))
      return fail(PROX_ERR_INVALID_ARG, "experts scales must be 4-byte aligned");
  }
  return PROX_OK;
}

// A product's arguments without the checks (the caller's own, or a layer's).
GroupedArgs grouped_args(const prox_experts* e, const void* a, int a_rows, int64_t a_stride, const float* a_scale,
                         const int32_t* row_index, const int32_t* offsets, int rows, void* out, int out_dtype,
                         int64_t out_stride) {
  const int es = elem(e->wdtype);
  GroupedArgs g;
  g.a = static_cast<const uint8_t*>(a);
  g.a_scale = a_scale;
  g.row_index = row_index;
  g.offsets = offsets;
  g.w = static_cast<const uint8_t*>(e->w);
  g.w_gate = static_cast<const uint8_t*>(e->w_gate);
  g.w_scale = e->w_scale;
  g.w_gate_scale = e->w_gate_scale;
  g.out = static_cast<uint8_t*>(out);
  g.a_stride = a_stride * es;
  g.w_stride = e->row_stride * es;
  g.w_group = e->group_stride * es;
  g.out_stride = out_stride * elem(out_dtype);
  g.a_rows = a_rows;
  g.rows = rows;
  g.n_groups = e->n_groups;
  g.n = e->n;
  g.kbytes = e->k * es;
  g.kblocks = blocks128(e->k);
  g.nblocks = blocks128(e->n);
  g.wdtype = e->wdtype;
  g.out_dtype = out_dtype;
  g.act = e->activation;
  return g;
}

prox_status check_route_shape(int32_t n_tokens, int32_t n_experts, int32_t top_k) {
  if (n_tokens < 0 || n_experts < 1 || top_k < 1)
    return fail(PROX_ERR_INVALID_ARG, "n_tokens %d, n_experts %d, top_k %d: need >= 0, >= 1, >= 1", n_tokens, n_experts,
                top_k);
  if (top_k > n_experts) return fail(PROX_ERR_INVALID_ARG, "top_k %d above n_experts %d", top_k, n_experts);
  if (n_experts > kMaxExperts || top_k > kMaxTopK)
    return fail(PROX_ERR_UNSUPPORTED, "n_experts %d above %d or top_k %d above %d", n_experts, kMaxExperts, top_k,
                kMaxTopK);
  if (static_cast<int64_t>(n_tokens) * top_k > kMaxRows)
    return fail(PROX_ERR_UNSUPPORTED, "n_tokens * top_k above 2^30");
  return PROX_OK;
}

// Workspace of prox_moe_ffn: byte offsets of its parts.
struct MoePlan {
  size_t logits, idx, weight, offsets, row_token, row_of, route, h, o, xq, xs, hq, hs, bytes;
};
MoePlan moe_plan(const prox_moe_layer* L, int tokens) {
  const int d = L->up.k, f = L->up.n;
  const size_t t = static_cast<size_t>(tokens), rows = t * L->top_k;
  const bool fp8 = L->up.wdtype == PROX_FP8;
  const size_t es = L->up.wdtype == PROX_F32 ? 4 : 2;
  size_t off = 0;
  auto part = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  MoePlan p;
  p.logits = part(t * L->up.n_groups * 4);
  p.idx = part(rows * 4);
  p.weight = part(rows * 4);
  p.offsets = part((static_cast<size_t>(L->up.n_groups) + 1) * 4);
  p.row_token = part(rows * 4);
  p.row_of = part(rows * 4);
  p.route = part(route_workspace(tokens, L->up.n_groups));
  p.h = part(rows * f * es);
  p.o = part(rows * d * es);
  p.xq = part(fp8 ? t * d : 0);
  p.xs = part(fp8 ? t * blocks128(d) * 4 : 0);
  p.hq = part(fp8 ? rows * f : 0);
  p.hs = part(fp8 ? rows * blocks128(f) * 4 : 0);
  p.bytes = off;
  return p;
}

prox_status check_moe(const prox_moe_layer* L, int32_t n_tokens) {
  if (!L) return fail(PROX_ERR_INVALID_ARG, "layer descriptor is NULL");
  prox_status st = check_experts(&L->up);
  if (st != PROX_OK) return st;
  if ((st = check_experts(&L->down)) != PROX_OK) return st;
  if (!L->up.w_gate || L->down.w_gate)
    return fail(PROX_ERR_INVALID_ARG, "layer up must be gated (w_gate) and down must not");
  if (L->up.n_groups != L->down.n_groups || L->up.n != L->down.k || L->up.k != L->down.n ||
      L->up.wdtype != L->down.wdtype)
    return fail(PROX_ERR_INVALID_ARG, "layer up [%d][%d][%d] and down [%d][%d][%d] (or their types) do not fit",
                L->up.n_groups, L->up.n, L->up.k, L->down.n_groups, L->down.n, L->down.k);
  if (L->reserved != 0 || (L->renormalize != 0 && L->renormalize != 1))
    return fail(PROX_ERR_INVALID_ARG, "layer renormalize must be 0 or 1 and reserved 0");
  const int es = L->up.wdtype == PROX_F32 ? 4 : 2;  // type of x, the router and the rows between the products
  if (L->up.k * es % 16 != 0 || L->up.n * es % 16 != 0)
    return fail(PROX_ERR_UNSUPPORTED, "layer d_model %d and d_ff %d must be multiples of 16 bytes", L->up.k, L->up.n);
  if (static_cast<int64_t>(L->up.k) * es >= kMaxWeightRow)  // a row of w_router, which may be wider than up's
    return fail(PROX_ERR_UNSUPPORTED, "layer d_model %d: rows of w_router must be below 8 MiB", L->up.k);
  if (!L->w_router || !aligned(L->w_router, 16))
    return fail(PROX_ERR_INVALID_ARG, "layer w_router must be non-NULL and 16-byte aligned");
  return check_route_shape(n_tokens, L->up.n_groups, L->top_k);
}

}  // namespace
}  // namespace prox

using namespace prox;

PROX_API prox_status prox_grouped_matmul(const prox_experts* e, const void* a, int32_t a_rows, int64_t a_stride,
                                         const float* a_scale, const int32_t* row_index, const int32_t* offsets,
                                         int32_t rows, void* out, int32_t out_dtype, int64_t out_stride, void* stream) {
  try {
    clear_error();
    prox_status st = check_experts(e);
    if (st != PROX_OK) return st;
    if (rows < 0 || rows > kMaxRows || a_rows < 0)
      return fail(PROX_ERR_INVALID_ARG, "rows %d outside [0, 2^30] or a_rows %d negative", rows, a_rows);
    if (out_dtype != PROX_F32 && out_dtype != PROX_BF16)
      return fail(PROX_ERR_INVALID_ARG, "out_dtype %d is neither PROX_F32 nor PROX_BF16", out_dtype);
    if (!offsets && e->n_groups != 1)
      return fail(PROX_ERR_INVALID_ARG, "offsets may be NULL for one group only (n_groups %d)", e->n_groups);
    if (!row_index && a_rows < rows)
      return fail(PROX_ERR_INVALID_ARG, "a_rows %d below rows %d without a row_index", a_rows, rows);
    const int es = elem(e->wdtype);
    if (a_stride < e->k || out_stride < e->n)
      return fail(PROX_ERR_INVALID_ARG, "a_stride below k or out_stride below n");
    if (a_stride > kMaxStride || out_stride > kMaxStride)
      return fail(PROX_ERR_UNSUPPORTED, "strides must be at most 2^40 elements");
    if (a_stride * es % 16 != 0) return fail(PROX_ERR_UNSUPPORTED, "a_stride must be a multiple of 16 bytes");
    if (rows == 0) return PROX_OK;
    if (a_rows == 0) return fail(PROX_ERR_INVALID_ARG, "a_rows is 0 with %d rows", rows);
    if (!a || !out || (e->wdtype == PROX_FP8 && !a_scale))
      return fail(PROX_ERR_INVALID_ARG, "a, out and (PROX_FP8) a_scale must be non-NULL");
    if (!aligned(a, 16) || !aligned(out, elem(out_dtype)) || !aligned(a_scale, 4) || !aligned(row_index, 4) ||
        !aligned(offsets, 4))
      return fail(PROX_ERR_INVALID_ARG, "a must be 16-byte aligned, out by its element, the others by 4 bytes");
    const hipError_t err = launch_grouped(grouped_args(e, a, a_rows, a_stride, a_scale, row_index, offsets, rows, out,
                                                       out_dtype, out_stride),
                                          device_cus(), static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return hip_fail(err, "grouped product launch");
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}

PROX_API prox_status prox_expert_route_workspace_size(int32_t n_tokens, int32_t n_experts, int32_t top_k,
                                                      size_t* bytes) {
  try {
    clear_error();
    if (!bytes) return fail(PROX_ERR_INVALID_ARG, "bytes is NULL");
    const prox_status st = check_route_shape(n_tokens, n_experts, top_k);
    if (st != PROX_OK) return st;
    *bytes = route_workspace(n_tokens, n_experts);
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}

PROX_API prox_status prox_expert_route(const void* logits, int32_t logits_dtype, int32_t n_tokens, int32_t n_experts,
                                       int32_t top_k, int32_t renormalize, int32_t* expert_idx, float* weight,
                                       int32_t* offsets, int32_t* row_token, int32_t* row_of, void* ws, size_t ws_bytes,
                                       void* stream) {
  try {
    clear_error();
    const prox_status st = check_route_shape(n_tokens, n_experts, top_k);
    if (st != PROX_OK) return st;
    if (logits_dtype != PROX_F32 && logits_dtype != PROX_BF16)
      return fail(PROX_ERR_INVALID_ARG, "logits_dtype %d is neither PROX_F32 nor PROX_BF16", logits_dtype);
    if (renormalize != 0 && renormalize != 1) return fail(PROX_ERR_INVALID_ARG, "renormalize must be 0 or 1");
    if (!offsets || !ws || (n_tokens > 0 && (!logits || !expert_idx || !weight || !row_token || !row_of)))
      return fail(PROX_ERR_INVALID_ARG, "logits, the outputs and ws must be non-NULL");
    if (!aligned(logits, elem(logits_dtype)) || !aligned(expert_idx, 4) || !aligned(weight, 4) ||
        !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(row_of, 4) || !aligned(ws, 256))
      return fail(PROX_ERR_INVALID_ARG, "logits and outputs must be aligned by their elements, ws by 256 bytes");
    const size_t need = route_workspace(n_tokens, n_experts);
    if (ws_bytes < need)
      return fail(PROX_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, need);
    RouteArgs r;
    r.logits = logits;
    r.logits_dtype = logits_dtype;
    r.tokens = n_tokens;
    r.experts = n_experts;
    r.top_k = top_k;
    r.renormalize = renormalize;
    r.expert_idx = expert_idx;
    r.weight = weight;
    r.offsets = offsets;
    r.row_token = row_token;
    r.row_of = row_of;
    r.block_count = static_cast<int*>(ws);
    const hipError_t err = launch_route(r, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return hip_fail(err, "route launch");
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}

PROX_API prox_status prox_fp8_quantize(const void* x, int32_t x_dtype, int32_t rows, int32_t k, int64_t x_stride,
                                       int32_t block_rows, void* q, int64_t q_stride, float* scale, void* stream) {
  try {
    clear_error();
    if (x_dtype != PROX_F32 && x_dtype != PROX_BF16)
      return fail(PROX_ERR_INVALID_ARG, "x_dtype %d is neither PROX_F32 nor PROX_BF16", x_dtype);
    if (rows < 0 || rows > kMaxRows || k < 1 || k > kMaxDim)
      return fail(PROX_ERR_INVALID_ARG, "rows %d outside [0, 2^30] or k %d outside [1, 2^24]", rows, k);
    if (block_rows != 1 && block_rows != kScaleBlock)
      return fail(PROX_ERR_INVALID_ARG, "block_rows %d is neither 1 nor 128", block_rows);
    if (x_stride < k || q_stride < k) return fail(PROX_ERR_INVALID_ARG, "x_stride or q_stride below k");
    if (x_stride > kMaxStride || q_stride > kMaxStride)
      return fail(PROX_ERR_UNSUPPORTED, "strides must be at most 2^40 elements");
    if (k % 16 != 0 || q_stride % 16 != 0 || x_stride * elem(x_dtype) % 16 != 0)
      return fail(PROX_ERR_UNSUPPORTED, "k must be a multiple of 16 and the strides multiples of 16 bytes");
    if (rows == 0) return PROX_OK;
    if (!x || !q || !scale) return fail(PROX_ERR_INVALID_ARG, "x, q and scale must be non-NULL");
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4))
      return fail(PROX_ERR_INVALID_ARG, "x and q must be 16-byte aligned, scale 4-byte aligned");
    QuantizeArgs a;
    a.x = static_cast<const uint8_t*>(x);
    a.q = static_cast<uint8_t*>(q);
    a.scale = scale;
    a.x_stride = x_stride * elem(x_dtype);
    a.q_stride = q_stride;
    a.x_dtype = x_dtype;
    a.rows = rows;
    a.k = k;
    a.block_rows = block_rows;
    const hipError_t err = launch_quantize(a, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return hip_fail(err, "quantize launch");
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}

namespace {
CombineArgs combine_args(const void* h, int h_dtype, int h_rows, int64_t h_stride, const int32_t* row_of,
                         const float* weight, int tokens, int top_k, int n, void* y, int y_dtype, int64_t y_stride) {
  CombineArgs a;
  a.h = static_cast<const uint8_t*>(h);
  a.row_of = row_of;
  a.weight = weight;
  a.y = static_cast<uint8_t*>(y);
  a.h_stride = h_stride * elem(h_dtype);
  a.y_stride = y_stride * elem(y_dtype);
  a.h_dtype = h_dtype;
  a.y_dtype = y_dtype;
  a.h_rows = h_rows;
  a.tokens = tokens;
  a.top_k = top_k;
  a.n = n;
  a.vec = aligned(h, 16) && aligned(y, 16) && a.h_stride % 16 == 0 && a.y_stride % 16 == 0 && n % 8 == 0;
  return a;
}
}  // namespace

PROX_API prox_status prox_expert_combine(const void* h, int32_t h_dtype, int32_t h_rows, int64_t h_stride,
                                         const int32_t* row_of, const float* weight, int32_t n_tokens, int32_t top_k,
                                         int32_t n, void* y, int32_t y_dtype, int64_t y_stride, void* stream) {
  try {
    clear_error();
    if ((h_dtype != PROX_F32 && h_dtype != PROX_BF16) || (y_dtype != PROX_F32 && y_dtype != PROX_BF16))
      return fail(PROX_ERR_INVALID_ARG, "h_dtype %d or y_dtype %d is neither PROX_F32 nor PROX_BF16", h_dtype, y_dtype);
    if (n_tokens < 0 || h_rows < 0 || top_k < 1 || top_k > kMaxTopK || n < 1 ||
        static_cast<int64_t>(n_tokens) * top_k > kMaxRows)
      return fail(PROX_ERR_INVALID_ARG, "n_tokens %d, h_rows %d, top_k %d (1..%d) or n %d out of range", n_tokens, h_rows,
                  top_k, kMaxTopK, n);
    if (h_stride < n || y_stride < n) return fail(PROX_ERR_INVALID_ARG, "h_stride or y_stride below n");
    if (n > kMaxDim || h_stride > kMaxStride || y_stride > kMaxStride)
      return fail(PROX_ERR_UNSUPPORTED, "n %d above 2^24, or strides above 2^40 elements", n);
    if (n_tokens == 0) return PROX_OK;
    if (!y || !row_of || !weight || (h_rows > 0 && !h))
      return fail(PROX_ERR_INVALID_ARG, "h, row_of, weight and y must be non-NULL");
    if (!aligned(h, elem(h_dtype)) || !aligned(y, elem(y_dtype)) || !aligned(row_of, 4) || !aligned(weight, 4))
      return fail(PROX_ERR_INVALID_ARG, "buffers must be aligned by their elements");
    const hipError_t err = launch_combine(combine_args(h, h_dtype, h_rows, h_stride, row_of, weight, n_tokens, top_k, n,
                                                       y, y_dtype, y_stride),
                                          static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return hip_fail(err, "combine launch");
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}

PROX_API prox_status prox_moe_workspace_size(const prox_moe_layer* layer, int32_t n_tokens, size_t* bytes) {
  try {
    clear_error();
    if (!bytes) return fail(PROX_ERR_INVALID_ARG, "bytes is NULL");
    const prox_status st = check_moe(layer, n_tokens);
    if (st != PROX_OK) return st;
    *bytes = moe_plan(layer, n_tokens).bytes;
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}

PROX_API prox_status prox_moe_ffn(const prox_moe_layer* L, const void* x, int32_t n_tokens, float* y, void* ws,
                                  size_t ws_bytes, void* stream) {
  try {
    clear_error();
    prox_status st = check_moe(L, n_tokens);
    if (st != PROX_OK) return st;
    if (n_tokens == 0) return PROX_OK;
    if (!x || !y || !ws) return fail(PROX_ERR_INVALID_ARG, "x, y and ws must be non-NULL");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 256))
      return fail(PROX_ERR_INVALID_ARG, "x and y must be 16-byte aligned, ws 256-byte aligned");
    const MoePlan p = moe_plan(L, n_tokens);
    if (ws_bytes < p.bytes)
      return fail(PROX_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes, p.bytes);
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(ws);
    const int d = L->up.k, f = L->up.n, rows = n_tokens * L->top_k, cus = device_cus();
    const bool fp8 = L->up.wdtype == PROX_FP8;
    const int xdtype = L->up.wdtype == PROX_F32 ? PROX_F32 : PROX_BF16;
    float* logits = reinterpret_cast<float*>(base + p.logits);
    int32_t* offsets = reinterpret_cast<int32_t*>(base + p.offsets);
    int32_t* row_token = reinterpret_cast<int32_t*>(base + p.row_token);
    int32_t* row_of = reinterpret_cast<int32_t*>(base + p.row_of);
    float* weight = reinterpret_cast<float*>(base + p.weight);
    // logits in fp32: the router's choice is not rounded to the layer's type
    prox_experts router = {};
    router.n_groups = 1;
    router.n = L->up.n_groups;
    router.k = d;
    router.wdtype = xdtype;
    router.row_stride = d;
    router.w = L->w_router;
    hipError_t e = launch_grouped(grouped_args(&router, x, n_tokens, d, nullptr, nullptr, nullptr, n_tokens, logits,
                                               PROX_F32, router.n),
                                  cus, s);
    if (e != hipSuccess) return hip_fail(e, "router product launch");
    RouteArgs r;
    r.logits = logits;
    r.logits_dtype = PROX_F32;
    r.tokens = n_tokens;
    r.experts = L->up.n_groups;
    r.top_k = L->top_k;
    r.renormalize = L->renormalize;
    r.expert_idx = reinterpret_cast<int32_t*>(base + p.idx);
    r.weight = weight;
    r.offsets = offsets;
    r.row_token = row_token;
    r.row_of = row_of;
    r.block_count = reinterpret_cast<int*>(base + p.route);
    if ((e = launch_route(r, s)) != hipSuccess) return hip_fail(e, "route launch");
    const void* a = x;
    float* xs = nullptr;
    auto quantize = [&](const void* src, int64_t n, int k, size_t q_at, size_t s_at) {
      QuantizeArgs q;
      q.x = static_cast<const uint8_t*>(src);
      q.q = base + q_at;
      q.scale = reinterpret_cast<float*>(base + s_at);
      q.x_stride = static_cast<int64_t>(k) * 2;
      q.q_stride = k;
      q.x_dtype = PROX_BF16;
      q.rows = static_cast<int>(n);
      q.k = k;
      q.block_rows = 1;
      return launch_quantize(q, s);
    };
    if (fp8) {
      if ((e = quantize(x, n_tokens, d, p.xq, p.xs)) != hipSuccess) return hip_fail(e, "quantize launch");
      a = base + p.xq;
      xs = reinterpret_cast<float*>(base + p.xs);
    }
    // the rows between the products are stored in x's type: half the traffic of
    // fp32 at one rounding of 2^-8 relative, as a layer of that type stores them
    void* h = base + p.h;
    e = launch_grouped(grouped_args(&L->up, a, n_tokens, d, xs, row_token, offsets, rows, h, xdtype, f), cus, s);
    if (e != hipSuccess) return hip_fail(e, "up/gate product launch");
    float* hs = nullptr;
    const void* hin = h;
    if (fp8) {
      if ((e = quantize(h, rows, f, p.hq, p.hs)) != hipSuccess) return hip_fail(e, "quantize launch");
      hin = base + p.hq;
      hs = reinterpret_cast<float*>(base + p.hs);
    }
    void* o = base + p.o;
    e = launch_grouped(grouped_args(&L->down, hin, rows, f, hs, nullptr, offsets, rows, o, xdtype, d), cus, s);
    if (e != hipSuccess) return hip_fail(e, "down product launch");
    e = launch_combine(combine_args(o, xdtype, rows, d, row_of, weight, n_tokens, L->top_k, d, y, PROX_F32, d), s);
    if (e != hipSuccess) return hip_fail(e, "combine launch");
    return PROX_OK;
  } catch (...) {
    return fail(PROX_ERR_INTERNAL, "unexpected exception");
  }
}
