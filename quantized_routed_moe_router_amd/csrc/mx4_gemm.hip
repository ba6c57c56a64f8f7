// Products of many rows of bf16 activations with 4-bit microscaled weights:
// the routed experts' gate/up and down products and the dense product.
//
// A workgroup of four waves takes up to 96 activation rows (one expert's
// tokens, or rows of a matrix) and 64 G weight rows.  Each wave owns 16 G weight
// rows: their codes go from memory to its registers, 16 bytes (one block of
// 32, one scale) per lane, and become exact bf16 operands there by one
// conversion instruction per pair, so a weight is read and converted once per
// workgroup.  The activations, which all four waves need, are staged in LDS
// 128 columns at a time by loads that bypass the registers.
// Lane (r, g) = (l % 16, l / 16) holds block g of a row's 128 columns; step j
// of 4 multiplies columns 32 g + 8 j .. + 7 of both operands, so the four
// steps cover the 128 in another order, the same for both.
//
// Memory answers later than a stage lasts, so codes are asked for two and three
// stages ahead and activations two (three buffers); loads are counted in
// order, so a wait for activations lets the later codes fly.
//
// 2048 tokens, 8 of 256 experts, H = 4096, I = 2048 (64 tokens an expert, a
// tile each): gate and up 710 us (0.77 Pflop/s), down 680, which goes over its
// codes once for each of the intermediate's two terms (0.8 Pflop/s of products
// issued); for an fp32 result, three terms, the whole takes 1.66 ms, not 1.38.
// With one term alone down took 398 us.  Without their products gate and up
// and one term of down take 577 and 348 us, without their loads 600 and 340:
// both are near what they cost alone, the matrix units are busy 45% of the
// time, and the clock falls under them (activations of zeros: 10% less time).
// Gate and up read 3.3 GB for 2.3 GB of codes and scales; the excess fits
// lines of scales that come again, which are asked for 16 bytes a row at a
// time, four stages apart (asking for 32 or 64 changed nothing: 742 us, 740).
// Asking for the next tile's codes ahead in L2 made gate and up 817 us; with
// activations two buffers deep instead of three the whole, with one term, took
// 1316 us and not 1117.
#include "mx4_dev.h"

namespace ds4 {

namespace {

constexpr int GM_ROWS = 96;              // activation rows of a tile
constexpr int GM_STAGE = GM_ROWS * 256;  // bytes of one stage: 128 bf16 columns

// what a workgroup multiplies
template <int G>
struct GemmTile {
  const uint8_t *w[G];         // codes of the wave's groups of 16 weight rows (wave-uniform)
  uint32_t wo[G];              // the row in them that this lane loads
  const uint8_t *srow;         // scales of row l of the 16 G
  int64_t K;
  int nblk, nst;               // blocks of 32 and stages of 128 columns
};

template <int G>
struct Codes {
  u4 c[G];
};

// EVEN: K is a multiple of 128, and no stage ends early
template <int G, bool EVEN>
__device__ __forceinline__ void load_codes(const GemmTile<G> &t, int st, Codes<G> &c) {
  const int blk = 4 * st + (threadIdx.x & 3);
  if (EVEN || 4 * st + 4 <= t.nblk) {
#pragma unroll
    for (int i = 0; i < G; ++i) c.c[i] = load16(t.w[i] + (t.wo[i] + (uint32_t)blk * 16u));
  } else {  // the last stage of a length that is no multiple of 128: zeros past the end
#pragma unroll
    for (int i = 0; i < G; ++i) {
      c.c[i] = u4{0, 0, 0, 0};
      if (blk < t.nblk) c.c[i] = load16(t.w[i] + (t.wo[i] + (uint32_t)blk * 16u));
    }
  }
}

// Activation rows 16 q + 4 wave + lane/16 of the tile go to LDS row by row,
// 256 bytes each.
template <int MT, bool EVEN>
__device__ __forceinline__ void load_rows(const uint8_t *const *rows, int64_t K, int st, char *lds) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = (lane & 15) ^ place16(4 * wave + (lane >> 4));
  const int64_t k = (int64_t)st * 128 + c * 8;
  char *const to = lds + 4 * wave * 256;
  if (EVEN || (int64_t)st * 128 + 128 <= K) {
#pragma unroll
    for (int q = 0; q < MT; ++q) load_lds16(rows[q] + k * 2, to + 16 * q * 256);
    return;
  }
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    if (k < K) load_lds16(rows[q] + k * 2, to + 16 * q * 256);
    else *reinterpret_cast<u4 *>(to + 16 * q * 256 + lane * 16) = u4{0, 0, 0, 0};
  }
}

// acc[i][m] += weight rows of group i times activation rows 16 m .. over the
// K columns.  lds: three stages, then 1 KB of scales per wave.
template <int G, int MT, bool EVEN>
__device__ __forceinline__ void gemm_columns(const GemmTile<G> &t, const uint8_t *const *rows, char *lds, f4 (&acc)[G][MT]) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char *const lsc = lds + 3 * GM_STAGE + wave * 1024;
  const int last = t.nst - 1;
  // scales of 512 columns of the wave's 16 G rows, one row per lane, turned in
  // LDS into one dword per lane and group: byte s is the lane's block of stage s
  u4 sc;
  uint32_t sd[G];
  auto turn_scales = [&]() {
    *reinterpret_cast<u4 *>(lsc + lane * 16) = transpose_bytes(sc);
    lds_order();
#pragma unroll
    for (int i = 0; i < G; ++i) sd[i] = *reinterpret_cast<const uint32_t *>(lsc + (16 * i + r) * 16 + 4 * g);
    lds_order();
  };
  Codes<G> c0, c1, c2, c3;  // stages s % 4, turned to the lanes' order one stage before they are used
  auto turn_codes = [&](Codes<G> &c) {
#pragma unroll
    for (int i = 0; i < G; ++i) c.c[i] = to_lanes(c.c[i]);
  };
  sc = scales16(t.srow, 0, t.nblk);
  load_rows<MT, EVEN>(rows, t.K, 0, lds);
  asm volatile("" ::: "memory");  // the waits count the loads issued after these
  load_codes<G, EVEN>(t, 0, c0);
  load_codes<G, EVEN>(t, min(1, last), c1);
  load_rows<MT, EVEN>(rows, t.K, min(1, last), lds + GM_STAGE);
  turn_codes(c0);
  turn_scales();
  wait_vm<G + MT>();
  barrier_keep_loads();
  int s = 0;
  const char *x = lds;             // this stage's buffer
  char *in = lds + 2 * GM_STAGE;   // the buffer that is filled
  char *const end = lds + 3 * GM_STAGE;
  // One stage: the rows two stages on and, at every other one, the codes of
  // two stages (adjacent halves of 128-byte lines), then the products.  Past
  // the end the last stage is loaded again: with no condition on the loads
  // every wait is for a fixed number of them.
  auto stage = [&](auto S, const Codes<G> &now, Codes<G> &next, Codes<G> &l0, Codes<G> &l1) {
    if (S == 0) sc = scales16(t.srow, min(s + 4, last / 4 * 4) * 4, t.nblk);
    load_rows<MT, EVEN>(rows, t.K, min(s + 2, last), in);
    asm volatile("" ::: "memory");
    if (S % 2 == 0) {
      load_codes<G, EVEN>(t, min(s + 2, last), l0);
      load_codes<G, EVEN>(t, min(s + 3, last), l1);
      asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf8 b[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        b[m] = *reinterpret_cast<const bf8 *>(x + (16 * m + r) * 256 + (((4 * g + j) ^ place16(r)) << 4));
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const bf8 a = codes_bf16(now.c[i][j], scale_float((sd[i] >> (8 * S)) & 255u));
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = mfma_bf16(a, b[m], acc[i][m]);
      }
    }
    if (S == 3) turn_scales();
    turn_codes(next);
    // the next stage's rows have landed; on their way may be the rows after
    // them and one pair of stages' codes
    wait_vm<2 * G + MT>();
    barrier_keep_loads();
    x = x + GM_STAGE == end ? lds : x + GM_STAGE;
    in = in + GM_STAGE == end ? lds : in + GM_STAGE;
    return ++s > last;
  };
  for (;;) {
    if (stage(std::integral_constant<int, 0>{}, c0, c1, c2, c3)) break;
    if (stage(std::integral_constant<int, 1>{}, c1, c2, c2, c3)) break;
    if (stage(std::integral_constant<int, 2>{}, c2, c3, c0, c1)) break;
    if (stage(std::integral_constant<int, 3>{}, c3, c0, c0, c1)) break;
  }
  wait_vm<0>();  // the last loads into LDS, before it is used again or released
  barrier_keep_loads();
}

// ... over `planes` terms of the activations, plane bytes apart
template <int G, int MT, bool EVEN>
__device__ __forceinline__ void gemm_tile(const GemmTile<G> &t, const uint8_t **rows, int planes, int64_t plane, char *lds,
                                          f4 (&acc)[G][MT]) {
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f4{0, 0, 0, 0};
  for (int q = 0; q < planes; ++q) {
    gemm_columns<G, MT, EVEN>(t, rows, lds, acc);
#pragma unroll
    for (int m = 0; m < MT; ++m) rows[m] += plane;
  }
}

// group i of the wave: 16 rows of the matrix (w, s) from row0 on
template <int G>
__device__ __forceinline__ void weight_rows(GemmTile<G> &t, int i, const uint8_t *w, const uint8_t *s, int64_t row0, int64_t N) {
  if (row0 >= N) row0 = 0;  // a group past the end: read, never stored
  t.w[i] = w + row0 * (t.K / 2);
  const int lane = threadIdx.x & 63, c = lane >> 2, r = lane & 15;  // rows of this lane's codes and scales
  t.wo[i] = (uint32_t)(row0 + c < N ? c : N - 1 - row0) * (uint32_t)(t.K / 2);
  if ((lane >> 4) % G == i) t.srow = s + (row0 + r < N ? row0 + r : N - 1) * (t.K / 32);
}

template <int G, int MT, int PL, bool EVEN>
__device__ __forceinline__ void gateup_tile(const Mx4Experts &p, const Mx4Tile &tl, int nb, char *lds) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int A = p.T * p.k;
  GemmTile<G> t;
  t.K = p.H;
  t.nblk = p.H / 32;
  t.nst = (t.nblk + 3) / 4;
  const int n0 = nb * 32 * G + wave * 8 * G;
  const int64_t eo = (int64_t)tl.e * p.I;
#pragma unroll
  for (int i = 0; i < G; ++i) {  // gate, then up
    const bool up = i >= G / 2;
    const uint8_t *w = (up ? p.up : p.gate) + eo * (p.H / 2), *s = (up ? p.up_s : p.gate_s) + eo * (p.H / 32);
    weight_rows(t, i, w, s, n0 + 16 * (i % (G / 2)), p.I);
  }
  const uint8_t *rows[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    const int row = 16 * q + 4 * wave + (lane >> 4);
    int a = p.perm[tl.p0 + (row < tl.n ? row : 0)];
    a = a < 0 ? 0 : a >= A ? A - 1 : a;
    rows[q] = (const uint8_t *)(p.x + (int64_t)(a / p.k) * p.ldx);
  }
  f4 acc[G][MT];
  gemm_tile<G, MT, EVEN>(t, rows, 1, 0, lds, acc);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = 16 * m + r;
    if (row >= tl.n) continue;
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
      const int n = n0 + 16 * i + 4 * g;
      if (n >= p.I) continue;
      const f4 u = acc[i][m], v = acc[G / 2 + i][m];
      store_terms<PL>(p.h + (int64_t)(tl.p0 + row) * p.I + n, (int64_t)A * p.I, silu_mul(u[0], v[0]), silu_mul(u[1], v[1]),
                      silu_mul(u[2], v[2]), silu_mul(u[3], v[3]));
    }
  }
}

template <int G, int MT, int PL, bool EVEN>
__device__ __forceinline__ void down_tile(const Mx4Experts &p, const Mx4Tile &tl, int nb, char *lds) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int A = p.T * p.k;
  GemmTile<G> t;
  t.K = p.I;
  t.nblk = p.I / 32;
  t.nst = (t.nblk + 3) / 4;
  const int n0 = nb * 64 * G + wave * 16 * G;
  const int64_t eo = (int64_t)tl.e * p.H;
#pragma unroll
  for (int i = 0; i < G; ++i)
    weight_rows(t, i, p.down + eo * (p.I / 2), p.down_s + eo * (p.I / 32), n0 + 16 * i, p.H);
  const uint8_t *rows[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    const int row = 16 * q + 4 * wave + (lane >> 4);
    rows[q] = (const uint8_t *)(p.h + (int64_t)(tl.p0 + (row < tl.n ? row : 0)) * p.I);
  }
  f4 acc[G][MT];
  gemm_tile<G, MT, EVEN>(t, rows, PL, (int64_t)A * p.I * 2, lds, acc);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = 16 * m + r;
    if (row >= tl.n) continue;
    const int a = p.perm[tl.p0 + row];
    if (a < 0 || a >= A) continue;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int n = n0 + 16 * i + 4 * g;
      if (n < p.H) *reinterpret_cast<f4 *>(p.ya + (int64_t)a * p.H + n) = acc[i][m];
    }
  }
}

// one instance per number of groups of 16 activation rows, so that a tile of
// 70 tokens multiplies 80 rows and not 96
#define BY_GROUPS(n, CALL)      \
  switch (((n) + 15) / 16) {    \
    case 1: CALL(1); break;     \
    case 2: CALL(2); break;     \
    case 3: CALL(3); break;     \
    case 4: CALL(4); break;     \
    case 5: CALL(5); break;     \
    default: CALL(6); break;    \
  }

template <int G, int PL, bool DOWN, bool EVEN>
__global__ __launch_bounds__(256, 2) void k_mx4_gemm_experts(Mx4Experts p, int nrows) {
  __shared__ __attribute__((aligned(16))) char lds[3 * GM_STAGE + 4096];
  int ti, nb;
  if (!tile_of(blockIdx.x, p.tiles->count, nrows, ti, nb)) return;
  const Mx4Tile tl = p.tiles->tile[ti];
#define UP(MT) gateup_tile<G, MT, PL, EVEN>(p, tl, nb, lds)
#define DN(MT) down_tile<G, MT, PL, EVEN>(p, tl, nb, lds)
  if constexpr (DOWN) BY_GROUPS(tl.n, DN)
  else BY_GROUPS(tl.n, UP)
#undef UP
#undef DN
}

// The list of tiles, experts ascending: one workgroup, a thread per expert.
__global__ __launch_bounds__(512) void k_mx4_plan(Mx4Experts p) {
  __shared__ int32_t sum[512];
  const int e = threadIdx.x, A = p.T * p.k;
  int n = 0, p0 = 0;
  if (e < p.E) {
    p0 = p.offsets[e];
    n = p.counts[e];
    if (p0 < 0 || p0 > A) n = 0;
    else if (n > A - p0) n = A - p0;
    if (n < 0) n = 0;
  }
  const int nt = (n + GM_ROWS - 1) / GM_ROWS;
  sum[e] = nt;
  __syncthreads();
  for (int o = 1; o < 512; o <<= 1) {
    const int v = e >= o ? sum[e - o] : 0;
    __syncthreads();
    sum[e] += v;
    __syncthreads();
  }
  if (e == 511) p.tiles->count = sum[511] < p.max_tiles ? sum[511] : p.max_tiles;
  for (int i = 0; i < nt; ++i) {
    const int at = sum[e] - nt + i;
    if (at < p.max_tiles) p.tiles->tile[at] = Mx4Tile{e, p0 + i * GM_ROWS, n - i * GM_ROWS < GM_ROWS ? n - i * GM_ROWS : GM_ROWS, 0};
  }
}

template <int G, int MT, bool YBF, bool EVEN>
__device__ __forceinline__ void product_tile(const Mx4Product &p, int64_t m0, int64_t n, int nb, char *lds) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  GemmTile<G> t;
  t.K = p.K;
  t.nblk = (int)(p.K / 32);
  t.nst = (t.nblk + 3) / 4;
  const int64_t n0 = (int64_t)nb * 64 * G + wave * 16 * G;
#pragma unroll
  for (int i = 0; i < G; ++i) weight_rows(t, i, p.w, p.ws, n0 + 16 * i, p.N);
  const uint8_t *rows[MT];
#pragma unroll
  for (int q = 0; q < MT; ++q) {
    const int64_t row = 16 * q + 4 * wave + (lane >> 4);
    rows[q] = (const uint8_t *)p.a + (m0 + (row < n ? row : 0)) * p.lda * 2;
  }
  f4 acc[G][MT];
  gemm_tile<G, MT, EVEN>(t, rows, 1, 0, lds, acc);
  const bool wide = wide_rows(p);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = 16 * m + r;
    if (row >= n) continue;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float v[4] = {acc[i][m][0], acc[i][m][1], acc[i][m][2], acc[i][m][3]};
      store_cols<YBF, 4>(p, wide, m0 + row, n0 + 16 * i + 4 * g, v);
    }
  }
}

template <int G, bool YBF, bool EVEN>
__global__ __launch_bounds__(256, 2) void k_mx4_gemm(Mx4Product p, int mtiles, int nrows) {
  __shared__ __attribute__((aligned(16))) char lds[3 * GM_STAGE + 4096];
  int ti, nb;
  if (!tile_of(blockIdx.x, mtiles, nrows, ti, nb)) return;
  const int64_t m0 = (int64_t)ti * GM_ROWS, n = p.M - m0 < GM_ROWS ? p.M - m0 : GM_ROWS;
#define CALL(MT) product_tile<G, MT, YBF, EVEN>(p, m0, n, nb, lds)
  BY_GROUPS((int)n, CALL)
#undef CALL
}

}  // namespace

int64_t mx4_max_tiles(int64_t A, int64_t E) { return A / GM_ROWS + (A < E ? A : E); }

// Weight rows per wave: 64, or 32 (gate and up together) or 16 where these
// would leave CUs without a workgroup.  The number of tiles is known on the
// device alone; every expert with tokens has one at least.
hipError_t launch_mx4_gemm_experts(const Mx4Experts &p, hipStream_t s) {
  auto rows = [&](int n, int per) { return (n + per - 1) / per; };
  const int64_t A = (int64_t)p.T * p.k, used = A < p.E ? A : p.E, tiles = A / GM_ROWS > used ? A / GM_ROWS : used;
  const bool gu_small = tiles * rows(p.I, 128) < 256, dn_small = tiles * rows(p.H, 256) < 256;
  hipLaunchKernelGGL(k_mx4_plan, dim3(1), dim3(512), 0, s, p);
  const bool hu = p.H % 128 != 0, iu = p.I % 128 != 0;
#define PICK(G, PL, D, U) (U ? k_mx4_gemm_experts<G, PL, D, false> : k_mx4_gemm_experts<G, PL, D, true>)
  auto up = p.y_bf16 ? (gu_small ? PICK(2, 2, false, hu) : PICK(4, 2, false, hu)) : (gu_small ? PICK(2, 3, false, hu) : PICK(4, 3, false, hu));
  auto down = p.y_bf16 ? (dn_small ? PICK(1, 2, true, iu) : PICK(4, 2, true, iu)) : (dn_small ? PICK(1, 3, true, iu) : PICK(4, 3, true, iu));
#undef PICK
  const int nu = rows(p.I, gu_small ? 64 : 128), nd = rows(p.H, dn_small ? 64 : 256);
  hipLaunchKernelGGL(up, dim3(tile_grid(p.max_tiles, nu)), dim3(256), 0, s, p, nu);
  hipLaunchKernelGGL(down, dim3(tile_grid(p.max_tiles, nd)), dim3(256), 0, s, p, nd);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm(const Mx4Product &p, hipStream_t s) {
  const int64_t mt = (p.M + GM_ROWS - 1) / GM_ROWS;
  const bool small = mt * ((p.N + 255) / 256) < 256, u = p.K % 128 != 0;
#define PICK(G, Y) (u ? k_mx4_gemm<G, Y, false> : k_mx4_gemm<G, Y, true>)
  auto f = p.y_bf16 ? (small ? PICK(1, true) : PICK(4, true)) : (small ? PICK(1, false) : PICK(4, false));
#undef PICK
  const int64_t nr = (p.N + (small ? 63 : 255)) / (small ? 64 : 256);
  hipLaunchKernelGGL(f, dim3(tile_grid(mt, nr)), dim3(256), 0, s, p, (int)mt, (int)nr);
  return hipGetLastError();
}

}  // namespace ds4
