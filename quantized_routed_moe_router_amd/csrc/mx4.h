// Launch wrappers of the expert gate and of the 4-bit microscaled operators
// (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ds4 {

// ---------------------------------------------------------------- gate
struct GateArgs {
  const void *logits;   // [T, ld] fp32 or bf16
  int64_t ld;
  const float *bias;    // [E] or null
  int32_t T, E, k, G, top_groups, group_rank, per;  // per = E / G
  uint32_t per_inv;     // ceil(2^20 / per): e / per = e * per_inv >> 20 for e < 512
  int32_t score;        // ds4moe_score
  bool renorm, bf16;
  float scale;
  int32_t *idx;         // [T,k]
  float *w;             // [T,k]
  int32_t *counts, *offsets, *perm;  // all set, or all null
  uint16_t *ccnt;       // [nchunk][E, to an even number] counts of a chunk (more than one chunk)
  uint16_t *lrank;      // [T*k] an assignment's rank among its expert's in the chunk
  int32_t chunk, nchunk;
};

struct GateGradArgs {
  const void *logits;
  int64_t ld;
  const float *bias;    // [E] or null
  const int32_t *idx;
  const float *dw;
  void *dl;
  int64_t ldd;
  int32_t T, E, k, score;
  bool renorm, bf16;
  float scale;
};

int gate_chunk(int64_t T);       // tokens per workgroup of the gate
int gate_chunks_max(int64_t T);  // the most workgroups for T tokens or fewer
hipError_t launch_gate(const GateArgs &a, hipStream_t s);
hipError_t launch_gate_backward(const GateGradArgs &a, hipStream_t s);

// ---------------------------------------------------------------- 4-bit microscaled values
hipError_t launch_mx4_quantize(uint8_t *codes, uint8_t *scales, const void *src, bool bf16, int64_t rows, int64_t cols,
                               int64_t ld, hipStream_t s);
hipError_t launch_mx4_dequantize(void *dst, bool bf16, int64_t ld, const uint8_t *codes, const uint8_t *scales,
                                 int64_t rows, int64_t cols, hipStream_t s);

// y[M,N] = a[M,K] w[N,K]^T
struct Mx4Product {
  void *y;
  int64_t ldy;
  bool y_bf16;
  const void *a;              // bf16 [M, lda], or codes [M, K/2]
  const uint8_t *a_scales;    // codes' scales [M, K/32], null for bf16
  int64_t lda;
  const uint8_t *w, *ws;      // codes [N, K/2], scales [N, K/32]
  int64_t M, N, K;
};
hipError_t launch_mx4_product(const Mx4Product &p, hipStream_t s);

// up to 96 tokens of one expert: positions p0 .. p0 + n - 1 of the permutation
struct Mx4Tile {
  int32_t e, p0, n, pad;
};
struct Mx4Tiles {
  int32_t count, pad[3];
  Mx4Tile tile[1];            // [count]
};

// The routed SwiGLU experts.
struct Mx4Experts {
  const uint8_t *gate, *gate_s, *up, *up_s, *down, *down_s;  // [E,I,H/2], [E,I,H/32], down [E,H,I/2], [E,H,I/32]
  const uint16_t *x;          // bf16 [T, ldx]
  int64_t ldx;
  int32_t T, H, I, E, k;
  const int32_t *idx, *counts, *offsets, *perm;
  const float *w;
  void *y;                    // [T,H]
  bool y_bf16;
  uint16_t *h;                // [planes][T*k][I] bf16 by position of the permutation
  float *ya;                  // [T*k][H] by assignment
  Mx4Tiles *tiles;
  int32_t max_tiles;
};
int64_t mx4_max_tiles(int64_t assignments, int64_t experts);
hipError_t launch_mx4_gemm_experts(const Mx4Experts &p, hipStream_t s);  // h and ya; more than a few tokens
hipError_t launch_mx4_gemm(const Mx4Product &p, hipStream_t s);          // bf16 activations, many rows
hipError_t launch_mx4_gemm4(const Mx4Product &p, hipStream_t s);         // 4-bit activations, many rows
constexpr int MX4_FEW = 16;       // tokens that the experts' kernels for few of them take
// Rows of a product that its kernels for few take.  The rule goes by rows
// alone, as measured at N = K = 4096: bf16 activations of 64 rows 23 us there,
// 25 in the tiled kernel; 4-bit ones of 64 rows 16 us, 10 in the tiled kernel,
// of 32 rows 10 in both.
constexpr int MX4_FEW_ROWS = 64, MX4_FEW_ROWS4 = 32;
constexpr int MX4_ONE = 4;   // tokens whose down projection adds the experts up itself
// bf16 terms that the SwiGLU intermediate is held in, however many tokens a
// call has: three, 24 bits, for an fp32 result, two, 16 bits, for a bf16 one
// (one term's rounding, 2^-8 of a value, adds as much to the result as the
// result's own: 2.3e-3 off the 64-bit values where two leave 1.7e-3)
inline int mx4_h_planes(bool y_bf16) { return y_bf16 ? 2 : 3; }
// Whether a call takes the experts' kernels for few tokens: few each, that is
// (16 tokens with 2 of 8 experts: 103 us there, 47 in the tiled kernels).
inline bool mx4_few(int64_t T, int64_t k, int64_t E) { return T <= MX4_ONE || (T <= MX4_FEW && T * k <= 2 * E); }
hipError_t launch_mx4_product_few(const Mx4Product &p, hipStream_t s);
hipError_t launch_mx4_experts_few(const Mx4Experts &p, hipStream_t s);  // h, then ya, or y for up to MX4_ONE tokens
hipError_t launch_mx4_experts(const Mx4Experts &p, hipStream_t s);

}  // namespace ds4
