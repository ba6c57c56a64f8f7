// C ABI of the expert gate and of the 4-bit microscaled operators: argument
// validation (host only, before any launch) and workspace layout.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/ds4moe.h"
#include "mx4.h"

using namespace ds4;

namespace {

constexpr int64_t kMaxTokens = 1 << 20;
constexpr int64_t kMaxDim = 1 << 24;

inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? DS4MOE_OK : DS4MOE_ERR_HIP; }
inline bool real_dtype(int32_t d) { return d == DS4MOE_F32 || d == DS4MOE_BF16; }
inline size_t elem(int32_t d) { return d == DS4MOE_BF16 ? 2 : 4; }

template <typename T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(reinterpret_cast<char *>(ws) + off);
}

int validate_gating(const ds4moe_gating *g) {
  if (!g) return DS4MOE_ERR_NULL;
  if (!real_dtype(g->logits_dtype)) return DS4MOE_ERR_DTYPE;
  if (g->n_experts < 1 || g->n_experts > 512) return DS4MOE_ERR_SHAPE;
  if (g->n_groups < 1 || g->n_groups > 64 || g->n_experts % g->n_groups) return DS4MOE_ERR_SHAPE;
  if (g->top_groups < 1 || g->top_groups > g->n_groups) return DS4MOE_ERR_SHAPE;
  if (g->top_k < 1 || g->top_k > 16 || g->top_k > g->top_groups * (g->n_experts / g->n_groups)) return DS4MOE_ERR_SHAPE;
  if (g->group_rank != 1 && g->group_rank != 2) return DS4MOE_ERR_SHAPE;
  if (g->score < DS4MOE_SCORE_SQRT_SOFTPLUS || g->score > DS4MOE_SCORE_SOFTMAX) return DS4MOE_ERR_SHAPE;
  if (g->renorm != 0 && g->renorm != 1) return DS4MOE_ERR_SHAPE;
  if (!isfinite(g->scale)) return DS4MOE_ERR_SHAPE;
  return DS4MOE_OK;
}

// idx stands in for a topk_idx that is not asked for
struct GateLayout {
  size_t idx, ccnt, lrank, total;
};

GateLayout gate_layout(const ds4moe_gating &g, int64_t T) {
  GateLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  L.idx = take(4 * (size_t)T * g.top_k);
  L.ccnt = take(2 * (size_t)gate_chunks_max(T) * ((g.n_experts + 1) & ~1));
  L.lrank = take(2 * (size_t)T * g.top_k);
  L.total = off;
  return L;
}

int validate_mx4(const ds4moe_mx4_dims *d) {
  if (!d) return DS4MOE_ERR_NULL;
  if (!real_dtype(d->y_dtype)) return DS4MOE_ERR_DTYPE;
  if (d->hidden < 32 || d->hidden > 65536 || d->hidden % 32) return DS4MOE_ERR_SHAPE;
  if (d->inter < 32 || d->inter > 65536 || d->inter % 32) return DS4MOE_ERR_SHAPE;
  if (d->n_experts < 1 || d->n_experts > 512) return DS4MOE_ERR_SHAPE;
  if (d->top_k < 1 || d->top_k > 16 || d->top_k > d->n_experts) return DS4MOE_ERR_SHAPE;
  return DS4MOE_OK;
}

struct Mx4Layout {
  size_t h, ya, tiles, total;
};

Mx4Layout mx4_layout(const ds4moe_mx4_dims &d, int64_t T) {
  Mx4Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  const size_t A = (size_t)T * d.top_k;
  L.h = take(2 * A * mx4_h_planes(d.y_dtype == DS4MOE_BF16) * d.inter);
  L.ya = take(4 * A * d.hidden);
  L.tiles = take(sizeof(Mx4Tiles) + sizeof(Mx4Tile) * (size_t)mx4_max_tiles((int64_t)A, d.n_experts));
  L.total = off;
  return L;
}

}  // namespace

extern "C" {

size_t ds4moe_gate_workspace_bytes(const ds4moe_gating *g, int32_t T) {
  if (validate_gating(g) != DS4MOE_OK || T < 0 || T > kMaxTokens) return 0;
  return T == 0 ? 256 : gate_layout(*g, T).total;
}

int ds4moe_gate(const ds4moe_gating *g, const void *logits, int64_t ld, const float *bias, int32_t T,
                ds4moe_routing *out, void *ws, size_t ws_bytes, void *stream) {
  const int st = validate_gating(g);
  if (st) return st;
  if (!out) return DS4MOE_ERR_NULL;
  if (T < 0 || T > kMaxTokens || ld < g->n_experts || ld > kMaxDim) return DS4MOE_ERR_SHAPE;
  if (out->logits) return DS4MOE_ERR_UNSUPPORTED;
  const bool perm = out->perm != nullptr;
  if (!aligned(bias, 4) || !aligned(out->topk_idx, 4) || !aligned(out->topk_w, 4) || !aligned(out->counts, 4) ||
      !aligned(out->offsets, 4) || !aligned(out->perm, 4))
    return DS4MOE_ERR_ALIGN;
  if (T == 0) return DS4MOE_OK;
  if ((out->counts != nullptr) != perm || (out->offsets != nullptr) != perm) return DS4MOE_ERR_NULL;
  if (!logits) return DS4MOE_ERR_NULL;
  if (!aligned(logits, elem(g->logits_dtype))) return DS4MOE_ERR_ALIGN;
  const GateLayout L = gate_layout(*g, T);
  if (!ws) return DS4MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return DS4MOE_ERR_ALIGN;
  if (ws_bytes < L.total) return DS4MOE_ERR_WORKSPACE;
  GateArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.T = T;
  a.E = g->n_experts;
  a.k = g->top_k;
  a.G = g->n_groups;
  a.top_groups = g->top_groups;
  a.group_rank = g->group_rank;
  a.per = a.E / a.G;
  a.per_inv = ((1u << 20) + a.per - 1) / a.per;
  a.score = g->score;
  a.renorm = g->renorm != 0;
  a.bf16 = g->logits_dtype == DS4MOE_BF16;
  a.scale = g->scale;
  a.idx = out->topk_idx ? out->topk_idx : at<int32_t>(ws, L.idx);
  a.w = out->topk_w;
  a.counts = out->counts;
  a.offsets = out->offsets;
  a.perm = out->perm;
  a.ccnt = at<uint16_t>(ws, L.ccnt);
  a.lrank = at<uint16_t>(ws, L.lrank);
  a.chunk = gate_chunk(T);
  a.nchunk = (T + a.chunk - 1) / a.chunk;
  return hip_status(launch_gate(a, (hipStream_t)stream));
}

int ds4moe_gate_backward(const ds4moe_gating *g, const void *logits, int64_t ld, const float *bias,
                         const int32_t *topk_idx, const float *d_topk_w, int32_t T, void *d_logits, int64_t ldd,
                         void *stream) {
  const int st = validate_gating(g);
  if (st) return st;
  if (T < 0 || T > kMaxTokens || ld < g->n_experts || ldd < g->n_experts || ld > kMaxDim || ldd > kMaxDim)
    return DS4MOE_ERR_SHAPE;
  if (T == 0) return DS4MOE_OK;
  if (!logits || !topk_idx || !d_topk_w || !d_logits) return DS4MOE_ERR_NULL;
  const size_t el = elem(g->logits_dtype);
  if (!aligned(logits, el) || !aligned(d_logits, el) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(d_topk_w, 4))
    return DS4MOE_ERR_ALIGN;
  GateGradArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.idx = topk_idx;
  a.dw = d_topk_w;
  a.dl = d_logits;
  a.ldd = ldd;
  a.T = T;
  a.E = g->n_experts;
  a.k = g->top_k;
  a.score = g->score;
  a.renorm = g->renorm != 0;
  a.bf16 = g->logits_dtype == DS4MOE_BF16;
  a.scale = g->scale;
  return hip_status(launch_gate_backward(a, (hipStream_t)stream));
}

int ds4moe_mx4_quantize(uint8_t *codes, uint8_t *scales, const void *src, int32_t src_dtype, int64_t rows,
                        int64_t cols, int64_t ld, void *stream) {
  if (!real_dtype(src_dtype)) return DS4MOE_ERR_DTYPE;
  if (rows < 0 || cols < 0 || cols >= ((int64_t)1 << 31) || rows > ((int64_t)1 << 40) || ld < cols ||
      ld > ((int64_t)1 << 40))
    return DS4MOE_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DS4MOE_OK;
  if (!codes || !scales || !src) return DS4MOE_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(src, elem(src_dtype))) return DS4MOE_ERR_ALIGN;
  return hip_status(
      launch_mx4_quantize(codes, scales, src, src_dtype == DS4MOE_BF16, rows, cols, ld, (hipStream_t)stream));
}

int ds4moe_mx4_dequantize(void *dst, int32_t dst_dtype, int64_t ld, const uint8_t *codes, const uint8_t *scales,
                          int64_t rows, int64_t cols, void *stream) {
  if (!real_dtype(dst_dtype)) return DS4MOE_ERR_DTYPE;
  if (rows < 0 || cols < 0 || cols >= ((int64_t)1 << 31) || rows > ((int64_t)1 << 40) || ld < cols ||
      ld > ((int64_t)1 << 40))
    return DS4MOE_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DS4MOE_OK;
  if (!codes || !scales || !dst) return DS4MOE_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(dst, elem(dst_dtype))) return DS4MOE_ERR_ALIGN;
  return hip_status(
      launch_mx4_dequantize(dst, dst_dtype == DS4MOE_BF16, ld, codes, scales, rows, cols, (hipStream_t)stream));
}

int ds4moe_mx4_matmul(void *y, int32_t y_dtype, int64_t ldy, const void *a, const uint8_t *a_scales, int32_t a_dtype,
                      int64_t lda, const uint8_t *w, const uint8_t *w_scales, int64_t M, int64_t N, int64_t K,
                      void *stream) {
  if (!real_dtype(y_dtype) || (a_dtype != DS4MOE_BF16 && a_dtype != DS4MOE_MX4)) return DS4MOE_ERR_DTYPE;
  if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim || K < 32 || K > kMaxDim || K % 32) return DS4MOE_ERR_SHAPE;
  if (ldy < N || ldy > ((int64_t)1 << 40)) return DS4MOE_ERR_SHAPE;
  if (a_dtype == DS4MOE_MX4 ? lda != K : lda < K || lda % 8 || lda > ((int64_t)1 << 40)) return DS4MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return DS4MOE_OK;
  if (!y || !a || !w || !w_scales) return DS4MOE_ERR_NULL;
  if ((a_dtype == DS4MOE_MX4) != (a_scales != nullptr)) return DS4MOE_ERR_NULL;
  if (!aligned(y, 16) || !aligned(a, 16) || !aligned(w, 16)) return DS4MOE_ERR_ALIGN;
  Mx4Product p{};
  p.y = y;
  p.ldy = ldy;
  p.y_bf16 = y_dtype == DS4MOE_BF16;
  p.a = a;
  p.a_scales = a_scales;
  p.lda = lda;
  p.w = w;
  p.ws = w_scales;
  p.M = M;
  p.N = N;
  p.K = K;
  return hip_status(launch_mx4_product(p, (hipStream_t)stream));
}

size_t ds4moe_mx4_workspace_bytes(const ds4moe_mx4_dims *dims, int32_t T) {
  if (validate_mx4(dims) != DS4MOE_OK || T < 0 || T > kMaxTokens) return 0;
  return T == 0 ? 256 : mx4_layout(*dims, T).total;
}

int ds4moe_mx4_experts(const ds4moe_mx4_dims *dims, const ds4moe_mx4_weights *w, const void *x, int64_t ldx, int32_t T,
                       const ds4moe_routing *routing, void *y, void *ws, size_t ws_bytes, void *stream) {
  const int st = validate_mx4(dims);
  if (st) return st;
  const ds4moe_mx4_dims &d = *dims;
  if (T < 0 || T > kMaxTokens || ldx < d.hidden || ldx % 8 || ldx > kMaxDim) return DS4MOE_ERR_SHAPE;
  if (!w || !routing) return DS4MOE_ERR_NULL;
  if (!w->gate || !w->gate_scales || !w->up || !w->up_scales || !w->down || !w->down_scales) return DS4MOE_ERR_NULL;
  if (!aligned(w->gate, 16) || !aligned(w->up, 16) || !aligned(w->down, 16)) return DS4MOE_ERR_ALIGN;
  if (T == 0) return DS4MOE_OK;
  if (!x || !y || !routing->topk_idx || !routing->topk_w || !routing->counts || !routing->offsets || !routing->perm)
    return DS4MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(routing->topk_idx, 4) || !aligned(routing->topk_w, 4) ||
      !aligned(routing->counts, 4) || !aligned(routing->offsets, 4) || !aligned(routing->perm, 4))
    return DS4MOE_ERR_ALIGN;
  const Mx4Layout L = mx4_layout(d, T);
  if (!ws) return DS4MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return DS4MOE_ERR_ALIGN;
  if (ws_bytes < L.total) return DS4MOE_ERR_WORKSPACE;
  Mx4Experts p{};
  p.gate = w->gate;
  p.gate_s = w->gate_scales;
  p.up = w->up;
  p.up_s = w->up_scales;
  p.down = w->down;
  p.down_s = w->down_scales;
  p.x = (const uint16_t *)x;
  p.ldx = ldx;
  p.T = T;
  p.H = d.hidden;
  p.I = d.inter;
  p.E = d.n_experts;
  p.k = d.top_k;
  p.idx = routing->topk_idx;
  p.counts = routing->counts;
  p.offsets = routing->offsets;
  p.perm = routing->perm;
  p.w = routing->topk_w;
  p.y = y;
  p.y_bf16 = d.y_dtype == DS4MOE_BF16;
  p.h = at<uint16_t>(ws, L.h);
  p.ya = at<float>(ws, L.ya);
  p.tiles = at<Mx4Tiles>(ws, L.tiles);
  p.max_tiles = (int32_t)mx4_max_tiles((int64_t)T * d.top_k, d.n_experts);
  return hip_status(launch_mx4_experts(p, (hipStream_t)stream));
}

}  // extern "C"
