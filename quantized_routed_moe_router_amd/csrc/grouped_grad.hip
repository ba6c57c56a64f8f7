// Gradients of the products grouped by expert, in bf16 or fp16 operands:
//   dx[p] = W_e^T dy[p]                 (the sum runs over W's rows)
//   dW_e  = sum_p dy[p] x[row(p)]^T     (the sum runs over the expert's rows)
//
// The forward kernel's tiles and stages, 64 terms of the sum at a time.  An
// operand whose rows are the terms lies across: W in dx, both in dW.  It is
// staged as it lies, 64 rows by the tile's columns, and turned on the way to
// the registers by the LDS' transposing read, which gives lane i of 16 the
// column i of four rows.
#include "grouped_dev.h"

namespace ds4 {

namespace {

// four rows of a staged operand at `at` (lane i of 16 points at row i / 4,
// columns 4 (i % 4) ..): lane i gets column i of them
__device__ __forceinline__ u2 read_turned(const char *at) {
  return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)at));
}

// Places of an operand that lies across: row j (term j) of 64, the tile's
// columns.  Tile m of a wave's groups of 16 columns has columns 32 (m / 2) +
// 8 a + 4 (m % 2) + b in the place 4 a + b, so that a lane's results of two
// tiles are 8 adjacent ones.  Chunk c of 16 bytes of row j goes to c ^ 4 (j % 4).
__device__ __forceinline__ int across_place(int row) { return (row & 3) << 2; }

// DW: dW (both operands across), otherwise dx (W across)
template <class OP, bool DW, int BM, int BN, int WM, int WN, int NB>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_grouped_grad(GroupedGrad p, int mtiles_dw, int ntiles) {
  constexpr int WAVES = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int STAGE = (BM + BN) * 128, DA = BM / 8 / WAVES, DB = BN / 8 / WAVES;
  constexpr int CA = BM / 8, CB = BN / 8;  // chunks of a row of an operand that lies across
  static_assert(BM >= 128 && BN >= 128 && MT % 2 == 0 && NT % 2 == 0, "places of chunks stay in the row");
  __shared__ __attribute__((aligned(16))) char lds[NB * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  Segment t;
  int64_t m0 = 0;  // dW: the tile's first row
  int nt;
  if (DW) {
    int mt;
    if (!place_tile<4>(blockIdx.x, p.E * mtiles_dw, ntiles, mt, nt)) return;
    t.e = mt / mtiles_dw;
    m0 = (int64_t)(mt - t.e * mtiles_dw) * BM;
    t.p0 = 0;
    t.n = p.P;
    if (p.offsets) {
      t.p0 = min(max(p.offsets[t.e], 0), p.P);
      t.n = max(min(max(p.offsets[t.e + 1], 0), p.P) - t.p0, 0);
    }
  } else {
    Finder<BM> f;
    const int mtiles = f.count(p.offsets, p.E, p.P);
    int mt;
    if (!place_tile<4>(blockIdx.x, mtiles, ntiles, mt, nt)) return;
    t = f.find(mt);
  }
  const int64_t n0 = (int64_t)nt * BN;
  if (!DW && t.e < 0) {
    zero_rows(p.out, p.o_type, p.ldo, t.p0, t.n, n0, min(n0 + BN, p.K));
    return;
  }
  const char *const zeros = (const char *)kZeros;
  const int64_t terms = DW ? t.n : p.N;
  const int last = (int)((terms + 63) / 64) - 1, edge = (int)(terms - (int64_t)last * 64);  // terms of the last stage

  // this lane's row and column of load q of an operand that lies across
  auto across_row = [&](int q, int chunks) { return (q * WAVES + wave) * (64 / chunks) + lane / chunks; };
  auto across_col = [&](int q, int chunks) { return ((lane % chunks) ^ across_place(across_row(q, chunks))) * 8; };

  const char *sa[DA], *sb[DB];
  int ca[DA], at_x[DB];
  if (!DW) {
#pragma unroll
    for (int q = 0; q < DA; ++q) {
      const int row = (q * WAVES + wave) * 8 + (lane >> 3);
      ca[q] = (lane & 7) ^ place8(row & 15);
      sa[q] = p.dy + (int64_t)(t.p0 + min(row, t.n - 1)) * p.lddy + ca[q] * 16;
    }
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const int64_t c = n0 + across_col(q, CB);
      sb[q] = c < p.K ? p.w + (((int64_t)t.e * p.N + across_row(q, CB)) * p.K + c) * 2 : nullptr;
    }
  } else {
#pragma unroll
    for (int q = 0; q < DA; ++q) {
      const int64_t c = m0 + across_col(q, CA);
      sa[q] = c < p.N ? p.dy + (int64_t)(t.p0 + across_row(q, CA)) * p.lddy + c * 2 : nullptr;
    }
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const int64_t c = n0 + across_col(q, CB);
      sb[q] = c < p.K ? p.x + c * 2 : nullptr;
    }
  }
  // dW: the rows of x of stage st, asked for a stage ahead of their use
  auto find_rows = [&](int st) {
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const int row = st * 64 + across_row(q, CB);
      at_x[q] = row < t.n ? row_of(p.perm, p.k_inv, p.T, p.k, t.p0 + row) : -1;
    }
  };
  auto load = [&](int st, char *to) {
    const bool short_ = st == last && edge < 64;
#pragma unroll
    for (int q = 0; q < DA; ++q) {
      const char *s;
      if (DW) s = sa[q] && !(short_ && across_row(q, CA) >= edge) ? sa[q] + (int64_t)st * 64 * p.lddy : zeros;
      else s = short_ && ca[q] * 8 >= edge ? zeros : sa[q] + (int64_t)st * 128;
      load_lds16(s, to + (q * WAVES + wave) * 1024);
    }
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const char *s;
      if (DW) s = sb[q] && at_x[q] >= 0 ? sb[q] + at_x[q] * p.ldx : zeros;
      else s = sb[q] && !(short_ && across_row(q, CB) >= edge) ? sb[q] + (int64_t)st * 128 * p.K : zeros;
      load_lds16(s, to + BM * 128 + (q * WAVES + wave) * 1024);
    }
    asm volatile("" ::: "memory");
    if (DW) find_rows(st + 1);
  };
  typename OP::Acc acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = typename OP::Acc{0, 0, 0, 0};

  // terms 32 h + 8 g .. + 7 of tile m of a wave whose columns begin at chunk c0
  auto across = [&](const char *x, int chunks, int c0, int m, int h) {
    const int j = 32 * h + 8 * g + (r >> 2);  // this lane's row of the first four
    const char *at = x + (j * chunks + ((c0 + 4 * (m >> 1) + (r & 3)) ^ across_place(j))) * 16 + 8 * (m & 1);
    const u2 lo = read_turned(at), hi = read_turned(at + 4 * chunks * 16);
    return u4{lo[0], lo[1], hi[0], hi[1]};
  };
  const int fa = (wm * 16 * MT + r) * 128, f0 = (g ^ place8(r)) * 16;
  if (DW) find_rows(0);
#pragma unroll
  for (int i = 0; i < NB - 1; ++i)
    if (i <= last) load(i, lds + i * STAGE);
  wait_vm<0>();
  barrier_keep_loads();
  const char *x = lds;
  char *in = lds + (NB - 1) * STAGE;
  for (int s = 0; s <= last; ++s) {
    if (s + NB - 1 <= last) load(s + NB - 1, in);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u4 a[MT], b[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) b[i] = across(x + BM * 128, CB, wn * 2 * NT, i, h);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        a[m] = DW ? across(x, CA, wm * 2 * MT, m, h) : *reinterpret_cast<const u4 *>(x + fa + m * 2048 + (f0 ^ 64 * h));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][m] = OP::mul(b[i], a[m], acc[i][m]);
    }
    wait_vm<0>();
    barrier_keep_loads();
    x = x + STAGE == lds + NB * STAGE ? lds : x + STAGE;
    in = in + STAGE == lds + NB * STAGE ? lds : in + STAGE;
  }

  const int64_t ld = DW ? p.K : p.ldo, base = DW ? (int64_t)t.e * p.N * p.K : 0;
  const bool wide = wide_rows(p.o_type, ld);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    int64_t row;
    if (DW) {
      row = m0 + wm * 16 * MT + 32 * (m >> 1) + 8 * (r >> 2) + 4 * (m & 1) + (r & 3);
      if (row >= p.N) continue;
    } else {
      const int at = wm * 16 * MT + 16 * m + r;
      if (at >= t.n) continue;
      row = t.p0 + at;
    }
#pragma unroll
    for (int i = 0; i < NT; i += 2) {
      const int64_t n = n0 + wn * 16 * NT + 16 * i + 8 * g;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[i + j / 4][m][j % 4];
      if (n < p.K) store_values<8>(p.out, p.o_type, base + row * ld + n, p.K - n, wide, v);
    }
  }
}

template <class OP>
hipError_t dx(const GroupedGrad &p, hipStream_t s) {
  constexpr int BM = 128, BN = 128;
  const int64_t mt = grouped_max_tiles<BM>(p.offsets, p.E, p.P), nt = (p.K + BN - 1) / BN;
  hipLaunchKernelGGL((k_grouped_grad<OP, false, BM, BN, 2, 2, 2>), dim3((unsigned)((mt * nt + 7) / 8 * 8)), dim3(256), 0, s, p, 0, (int)nt);
  return hipGetLastError();
}
template <class OP>
hipError_t dw(const GroupedGrad &p, hipStream_t s) {
  constexpr int BM = 128, BN = 128;
  const int64_t mt = (p.N + BM - 1) / BM, nt = (p.K + BN - 1) / BN;
  hipLaunchKernelGGL((k_grouped_grad<OP, true, BM, BN, 2, 2, 2>), dim3((unsigned)((p.E * mt * nt + 7) / 8 * 8)), dim3(256), 0, s, p, (int)mt, (int)nt);
  return hipGetLastError();
}

// ---------------------------------------------------------------- gradients of shared rows
__global__ __launch_bounds__(256) void k_grouped_no_places(int32_t *places, int A) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < A) places[i] = -1;
}
// An assignment that stands twice counts with its last position: the same one every time.
__global__ __launch_bounds__(256) void k_grouped_places(int32_t *places, const int32_t *perm, int P, int A) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= P) return;
  const int a = perm[i];
  if (a >= 0 && a < A) atomicMax(places + a, i);
}

// dx[t] = sum over j of the rows of its assignments, in the order of j, in fp32 with one rounding
template <int NV>
__global__ __launch_bounds__(256) void k_grouped_add_up(void *dx, int64_t ldo, int o_type, const float *rows, const int32_t *places, int T, int k, int64_t K) {
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * NV;
  if (c >= K) return;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float v[NV] = {};
    for (int j = 0; j < k; ++j) {
      const int at = places[t * k + j];
      if (at < 0) continue;
#pragma unroll
      for (int i = 0; i < NV; i += 4) {
        const f4 u = *reinterpret_cast<const f4 *>(rows + at * K + c + i);
#pragma unroll
        for (int l = 0; l < 4; ++l) v[i + l] += u[l];
      }
    }
    store_values<NV>(dx, o_type, t * ldo + c, K - c, wide_rows(o_type, ldo), v);
  }
}

}  // namespace

hipError_t launch_grouped_dx(const GroupedGrad &p, hipStream_t s) { return p.type == DS4MOE_BF16 ? dx<OpBf16>(p, s) : dx<OpF16>(p, s); }
hipError_t launch_grouped_dw(const GroupedGrad &p, hipStream_t s) { return p.type == DS4MOE_BF16 ? dw<OpBf16>(p, s) : dw<OpF16>(p, s); }

hipError_t launch_grouped_places(int32_t *places, const int32_t *perm, int32_t P, int32_t A, hipStream_t s) {
  hipLaunchKernelGGL(k_grouped_no_places, dim3((A + 255) / 256), dim3(256), 0, s, places, A);
  if (P) hipLaunchKernelGGL(k_grouped_places, dim3((P + 255) / 256), dim3(256), 0, s, places, perm, P, A);
  return hipGetLastError();
}

hipError_t launch_grouped_add_up(void *dx, int64_t ldo, int32_t o_type, const float *rows, const int32_t *places, int32_t T, int32_t k,
                                 int64_t K, hipStream_t s) {
  hipLaunchKernelGGL(k_grouped_add_up<8>, dim3((unsigned)(T < (1 << 20) ? T : 1 << 20), (unsigned)((K + 2047) / 2048)), dim3(256), 0, s, dx, ldo,
                     o_type, rows, places, T, k, K);
  return hipGetLastError();
}

}  // namespace ds4
