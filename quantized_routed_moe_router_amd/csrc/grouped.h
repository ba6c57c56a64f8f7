// Launch wrappers of the products grouped by expert, their gradients and the
// 8-bit integer operators (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ds4 {

constexpr int GROUPED_EXPERTS = 512;  // the most experts (eight per lane of the wave that looks for a tile)

// y[p] = W_e x[row(p)] for offsets[e] <= p < offsets[e+1], or W_e^T x[row(p)]
// (turned: the gradient of the rows)
struct Grouped {
  void *y;                    // [P, ldy]
  int64_t ldy;                // elements
  int32_t y_type;             // ds4moe_dtype: fp32, bf16 or fp16
  int32_t type;               // of the operands: bf16, fp16 or 8-bit integers
  const char *x;              // rows of Kb bytes
  int64_t ldx;                // bytes
  const char *w;              // [E][N] rows of Kb bytes; turned: [E][Kb / 2] rows of N values of 16 bits
  bool turned;
  const float *xs, *ws;       // scales [T] and [E, N] of 8-bit operands
  const int32_t *offsets;     // [E + 1], or null: one group of all rows
  const int32_t *perm;        // [P]: row perm[p] / k, or null: row p
  int32_t E, k, P, T;
  uint32_t k_inv;             // ceil(2^31 / k)
  int64_t N, Kb;
  int32_t *places;            // turned: this many of them are set to -1 on the way
  int32_t n_places;
};
hipError_t launch_grouped(const Grouped &p, hipStream_t s);
hipError_t launch_grouped_few(const Grouped &p, hipStream_t s);

// dW_e = sum over p of dy[p] x[row(p)]^T
struct GroupedDw {
  void *dw;                   // [E, N, K]
  int32_t dw_type, type;
  const char *dy;             // [P] rows of N values
  int64_t lddy;               // bytes
  const char *x;              // rows of K values
  int64_t ldx;                // bytes
  const int32_t *offsets, *perm;
  int32_t E, k, P, T;
  uint32_t k_inv;
  int64_t N, K;
};
hipError_t launch_grouped_dw(const GroupedDw &p, hipStream_t s);

// Where the assignments of tokens stand: a list of the positions of each, those that have an expert
struct GroupedPlaces {
  int32_t *place;  // [A]: the first of the list, marked where there are more; -1 before and where there is none
  int32_t *next;   // [P]: what follows in the list, or -1
  const int32_t *perm, *offsets;
  int32_t E, P, A;
};
// the lists (P = 0: none, and nothing has to be -1 before)
hipError_t launch_grouped_places(const GroupedPlaces &q, hipStream_t s);
// dx[t] = sum over j of the rows of assignment t k + j, in the order of j and of the positions
hipError_t launch_grouped_add_up(void *dx, int64_t ldo, int32_t o_type, const float *rows, const GroupedPlaces &q,
                                 int32_t T, int32_t k, int64_t K, hipStream_t s);

// ---------------------------------------------------------------- 8-bit integers
hipError_t launch_int8_quantize(int8_t *codes, float *scales, const void *src, int32_t type, int64_t rows, int64_t cols,
                                int64_t ld, hipStream_t s);
hipError_t launch_int8_dequantize(void *dst, int32_t type, int64_t ld, const int8_t *codes, const float *scales,
                                  int64_t rows, int64_t cols, hipStream_t s);

// the dense product g of M rows (g.P) that are quantised on the way: a, rows lda values apart; g.x and g.xs are not read
bool int8_few_fits(int64_t M, int64_t K);
hipError_t launch_int8_few(const Grouped &g, const void *a, int32_t a_type, int64_t lda, int64_t K, hipStream_t s);

}  // namespace ds4
