// C ABI of the products grouped by expert, their gradients and the 8-bit
// integer operators: argument validation (host only, before any launch) and
// workspace layout.
#include <hip/hip_runtime.h>

#include "../../include/ds4moe.h"
#include "grouped.h"

using namespace ds4;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;    // of a dense product
constexpr int64_t kMaxGrouped = (int64_t)1 << 23;  // positions and tokens: entries of a permutation stay below 2^27
constexpr int64_t kMaxDim = 65536;
constexpr int64_t kMaxOut = (int64_t)1 << 37;  // values of a matrix: launches have less than 2^32 threads
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int64_t kMaxRow = (int64_t)1 << 22;  // values from row to row of an operand
constexpr int64_t kMaxSum8 = 131056;  // columns of 8-bit products: their sums stay in 32 bits at 128 x 128 a product

inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? DS4MOE_OK : DS4MOE_ERR_HIP; }
inline bool real_dtype(int32_t d) { return d == DS4MOE_F32 || d == DS4MOE_BF16 || d == DS4MOE_F16; }
inline bool half_dtype(int32_t d) { return d == DS4MOE_BF16 || d == DS4MOE_F16; }
inline int64_t elem(int32_t d) { return d == DS4MOE_F32 ? 4 : d == DS4MOE_I8 ? 1 : 2; }
inline uint32_t inverse(int32_t k) { return (uint32_t)((((uint64_t)1 << 31) + k - 1) / k); }

int validate_grouped(const ds4moe_grouped_dims *d) {
  if (!d) return DS4MOE_ERR_NULL;
  if (!half_dtype(d->dtype) && d->dtype != DS4MOE_I8) return DS4MOE_ERR_DTYPE;
  if (!real_dtype(d->y_dtype)) return DS4MOE_ERR_DTYPE;
  if (d->n_experts < 1 || d->n_experts > GROUPED_EXPERTS) return DS4MOE_ERR_SHAPE;
  if (d->top_k < 1 || d->top_k > 16) return DS4MOE_ERR_SHAPE;
  if (d->rows < 0 || d->rows > kMaxGrouped || d->tokens < 0 || d->tokens > kMaxGrouped) return DS4MOE_ERR_SHAPE;
  if (d->N < 1 || d->N > kMaxDim || d->K < 1 || d->K > kMaxDim) return DS4MOE_ERR_SHAPE;
  if (d->K * elem(d->dtype) % 16) return DS4MOE_ERR_SHAPE;
  if (d->rows * d->N > kMaxOut || d->rows * d->K > kMaxOut || d->n_experts * d->N * d->K > kMaxOut) return DS4MOE_ERR_SHAPE;
  return DS4MOE_OK;
}
int validate_grad(const ds4moe_grouped_dims *d) {
  const int st = validate_grouped(d);
  if (st) return st;
  if (!half_dtype(d->dtype)) return DS4MOE_ERR_UNSUPPORTED;
  return d->N % 8 ? DS4MOE_ERR_SHAPE : DS4MOE_OK;
}
// rows of `cols` values of operands, ld apart: 256 of them are within 32-bit offsets
inline bool row_step(int64_t ld, int64_t cols, int32_t dtype) { return ld >= cols && ld <= kMaxRow && ld * elem(dtype) % 16 == 0; }

struct DxLayout {
  size_t rows, next, places, total;
};
DxLayout dx_layout(const ds4moe_grouped_dims &d) {
  DxLayout L{};
  L.rows = 0;
  L.next = align256(4 * (size_t)d.rows * (size_t)d.K);
  L.places = L.next + align256(4 * (size_t)d.rows);
  L.total = L.places + align256(4 * (size_t)d.tokens * (size_t)d.top_k);
  return L;
}

}  // namespace

extern "C" {

int ds4moe_grouped_matmul(const ds4moe_grouped_dims *dims, void *y, int64_t ldy, const void *x, int64_t ldx,
                          const float *x_scales, const void *w, const float *w_scales, const int32_t *offsets,
                          const int32_t *perm, void *stream) {
  const int st = validate_grouped(dims);
  if (st) return st;
  const ds4moe_grouped_dims &d = *dims;
  if (ldy < d.N || ldy > kMaxLd || !row_step(ldx, d.K, d.dtype)) return DS4MOE_ERR_SHAPE;
  if (!perm && d.rows > d.tokens) return DS4MOE_ERR_SHAPE;
  if (d.rows == 0) return DS4MOE_OK;
  if (!y || !x || !w || !offsets) return DS4MOE_ERR_NULL;
  if ((d.dtype == DS4MOE_I8) != (x_scales != nullptr) || (d.dtype == DS4MOE_I8) != (w_scales != nullptr)) return DS4MOE_ERR_NULL;
  if (!aligned(y, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(offsets, 4) || !aligned(perm, 4))
    return DS4MOE_ERR_ALIGN;
  Grouped p{};
  p.y = y;
  p.ldy = ldy;
  p.y_type = d.y_dtype;
  p.type = d.dtype;
  p.x = (const char *)x;
  p.ldx = ldx * elem(d.dtype);
  p.w = (const char *)w;
  p.xs = x_scales;
  p.ws = w_scales;
  p.offsets = offsets;
  p.perm = perm;
  p.E = d.n_experts;
  p.k = d.top_k;
  p.P = (int32_t)d.rows;
  p.T = (int32_t)d.tokens;
  p.k_inv = inverse(d.top_k);
  p.N = d.N;
  p.Kb = d.K * elem(d.dtype);
  return hip_status(launch_grouped(p, (hipStream_t)stream));
}

size_t ds4moe_grouped_workspace_bytes(const ds4moe_grouped_dims *dims) {
  if (validate_grad(dims) != DS4MOE_OK) return 0;
  const size_t n = dx_layout(*dims).total;
  return n > 256 ? n : 256;
}

int ds4moe_grouped_dx(const ds4moe_grouped_dims *dims, void *dx, int64_t lddx, const void *dy, int64_t lddy, const void *w,
                      const int32_t *offsets, const int32_t *perm, void *ws, size_t ws_bytes, void *stream) {
  const int st = validate_grad(dims);
  if (st) return st;
  const ds4moe_grouped_dims &d = *dims;
  if (lddx < d.K || lddx > kMaxLd || !row_step(lddy, d.N, d.dtype)) return DS4MOE_ERR_SHAPE;
  if (!perm && d.rows != d.tokens) return DS4MOE_ERR_SHAPE;
  if (d.tokens == 0) return DS4MOE_OK;
  if (!dx || !w || !offsets || (d.rows && !dy)) return DS4MOE_ERR_NULL;
  if (!aligned(dx, 16) || !aligned(dy, 16) || !aligned(w, 16) || !aligned(offsets, 4) || !aligned(perm, 4))
    return DS4MOE_ERR_ALIGN;
  const DxLayout L = dx_layout(d);
  if (perm) {
    if (!ws) return DS4MOE_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return DS4MOE_ERR_ALIGN;
    if (ws_bytes < L.total) return DS4MOE_ERR_WORKSPACE;
  }
  const hipStream_t s = (hipStream_t)stream;
  float *const rows = reinterpret_cast<float *>((char *)ws + L.rows);
  const GroupedPlaces places{reinterpret_cast<int32_t *>((char *)ws + L.places), reinterpret_cast<int32_t *>((char *)ws + L.next),
                             perm, offsets, d.n_experts, (int32_t)d.rows, (int32_t)(d.tokens * d.top_k)};
  Grouped p{};
  p.y = perm ? rows : dx;
  p.ldy = perm ? d.K : lddx;
  p.y_type = perm ? DS4MOE_F32 : d.y_dtype;
  p.type = d.dtype;
  p.x = (const char *)dy;
  p.ldx = lddy * elem(d.dtype);
  p.w = (const char *)w;
  p.turned = true;
  p.offsets = offsets;
  p.E = d.n_experts;
  p.k = 1;
  p.P = p.T = (int32_t)d.rows;
  p.N = d.K;
  p.Kb = d.N * elem(d.dtype);
  p.places = perm ? places.place : nullptr;
  p.n_places = perm ? places.A : 0;
  hipError_t e = hipSuccess;
  if (d.rows) e = launch_grouped(p, s);
  if (e != hipSuccess || !perm) return hip_status(e);
  e = launch_grouped_places(places, s);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(launch_grouped_add_up(dx, lddx, d.y_dtype, rows, places, (int32_t)d.tokens, d.top_k, d.K, s));
}

int ds4moe_grouped_dw(const ds4moe_grouped_dims *dims, void *dw, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                      const int32_t *offsets, const int32_t *perm, void *stream) {
  const int st = validate_grad(dims);
  if (st) return st;
  const ds4moe_grouped_dims &d = *dims;
  if (!row_step(lddy, d.N, d.dtype) || !row_step(ldx, d.K, d.dtype)) return DS4MOE_ERR_SHAPE;
  if (!perm && d.rows > d.tokens) return DS4MOE_ERR_SHAPE;
  if (!dw || !offsets || (d.rows && (!dy || !x))) return DS4MOE_ERR_NULL;
  if (!aligned(dw, 16) || !aligned(dy, 16) || !aligned(x, 16) || !aligned(offsets, 4) || !aligned(perm, 4))
    return DS4MOE_ERR_ALIGN;
  GroupedDw p{};
  p.dw = dw;
  p.dw_type = d.y_dtype;
  p.type = d.dtype;
  p.dy = (const char *)dy;
  p.lddy = lddy * elem(d.dtype);
  p.x = (const char *)x;
  p.ldx = ldx * elem(d.dtype);
  p.offsets = offsets;
  p.perm = perm;
  p.E = d.n_experts;
  p.k = d.top_k;
  p.P = (int32_t)d.rows;
  p.T = (int32_t)d.tokens;
  p.k_inv = inverse(d.top_k);
  p.N = d.N;
  p.K = d.K;
  return hip_status(launch_grouped_dw(p, (hipStream_t)stream));
}

int ds4moe_int8_quantize(int8_t *codes, float *scales, const void *src, int32_t src_dtype, int64_t rows, int64_t cols,
                         int64_t ld, void *stream) {
  if (!real_dtype(src_dtype)) return DS4MOE_ERR_DTYPE;
  if (rows < 0 || cols < 0 || cols >= ((int64_t)1 << 31) || rows > ((int64_t)1 << 40) || ld < cols || ld > kMaxLd)
    return DS4MOE_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DS4MOE_OK;
  if (!codes || !scales || !src) return DS4MOE_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(src, elem(src_dtype))) return DS4MOE_ERR_ALIGN;
  return hip_status(launch_int8_quantize(codes, scales, src, src_dtype, rows, cols, ld, (hipStream_t)stream));
}

int ds4moe_int8_dequantize(void *dst, int32_t dst_dtype, int64_t ld, const int8_t *codes, const float *scales,
                           int64_t rows, int64_t cols, void *stream) {
  if (!real_dtype(dst_dtype)) return DS4MOE_ERR_DTYPE;
  if (rows < 0 || cols < 0 || cols >= ((int64_t)1 << 31) || rows > ((int64_t)1 << 40) || ld < cols || ld > kMaxLd)
    return DS4MOE_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DS4MOE_OK;
  if (!codes || !scales || !dst) return DS4MOE_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(dst, elem(dst_dtype))) return DS4MOE_ERR_ALIGN;
  return hip_status(launch_int8_dequantize(dst, dst_dtype, ld, codes, scales, rows, cols, (hipStream_t)stream));
}

size_t ds4moe_int8_workspace_bytes(int64_t M, int64_t K, int32_t a_dtype) {
  if (M < 0 || M > kMaxRows || K < 1 || K > kMaxSum8 || (!real_dtype(a_dtype) && a_dtype != DS4MOE_I8)) return 0;
  if (a_dtype == DS4MOE_I8 || M == 0) return 256;
  return align256((size_t)M * (size_t)((K + 15) / 16 * 16)) + align256(4 * (size_t)M);
}

int ds4moe_int8_matmul(void *y, int32_t y_dtype, int64_t ldy, const void *a, const float *a_scales, int32_t a_dtype,
                       int64_t lda, const int8_t *w, const float *w_scales, int64_t M, int64_t N, int64_t K, void *ws,
                       size_t ws_bytes, void *stream) {
  const bool codes = a_dtype == DS4MOE_I8;
  if (!real_dtype(y_dtype) || (!codes && !real_dtype(a_dtype))) return DS4MOE_ERR_DTYPE;
  if (M < 0 || N < 0 || M > kMaxRows || N > kMaxRows || K < 1 || K > kMaxSum8) return DS4MOE_ERR_SHAPE;
  if (M * N > kMaxOut || ldy < N || ldy > kMaxLd || lda < K || lda > (codes ? kMaxRow : kMaxLd)) return DS4MOE_ERR_SHAPE;
  if (codes && (K % 16 || lda % 16)) return DS4MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return DS4MOE_OK;
  if (!y || !a || !w || !w_scales) return DS4MOE_ERR_NULL;
  if (codes != (a_scales != nullptr)) return DS4MOE_ERR_NULL;
  if (!aligned(y, 16) || !aligned(a, codes ? 16 : elem(a_dtype)) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4))
    return DS4MOE_ERR_ALIGN;
  const int64_t K16 = (K + 15) / 16 * 16;
  Grouped p{};
  p.y = y;
  p.ldy = ldy;
  p.y_type = y_dtype;
  p.type = DS4MOE_I8;
  p.x = (const char *)a;
  p.ldx = lda;
  p.xs = a_scales;
  p.w = (const char *)w;
  p.ws = w_scales;
  p.E = p.k = 1;
  p.P = p.T = (int32_t)M;
  p.N = N;
  p.Kb = K16;
  const hipStream_t s = (hipStream_t)stream;
  if (!codes) {
    if (!ws) return DS4MOE_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return DS4MOE_ERR_ALIGN;
    if (ws_bytes < ds4moe_int8_workspace_bytes(M, K, a_dtype)) return DS4MOE_ERR_WORKSPACE;
    if (int8_few_fits(M, K)) return hip_status(launch_int8_few(p, a, a_dtype, lda, K, s));
    int8_t *const c = (int8_t *)ws;
    float *const sc = reinterpret_cast<float *>((char *)ws + align256((size_t)(M * K16)));
    const hipError_t e = launch_int8_quantize(c, sc, a, a_dtype, M, K, lda, s);
    if (e != hipSuccess) return hip_status(e);
    p.x = (const char *)c;
    p.ldx = K16;
    p.xs = sc;
  }
  return hip_status(launch_grouped(p, s));
}

}  // extern "C"
