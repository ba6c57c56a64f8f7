// Gradients of the products grouped by expert: of the weights,
//   dW_e = sum over p of dy[p] x[row(p)]^T,
// in bf16 or fp16 operands, and the sum of the gradients of rows that several
// experts share.  (The gradient of the rows is a product by turned weights.)
//
// A workgroup of WN waves has 16 MT rows and 32 WN columns of one dW_e, 64
// terms of the sum at a time.  Both operands lie across.
#include "grouped_dev.h"

namespace ds4 {

namespace {

// FAR: rows of x that 32-bit offsets do not reach
template <class OP, int WN, int MT, bool FAR>
__global__ __launch_bounds__(64 * WN, 2) void k_grouped_dw(GroupedDw p, int mtiles, int ntiles) {
  constexpr int NT = 2, DA = 2 * MT / WN, DB = 4, CA = 2 * MT, CB = 4 * WN;  // loads per wave; chunks of a staged row
  constexpr int BOFF = DA * WN * 1024, STAGE = BOFF + DB * WN * 1024;
  static_assert(DA * WN == 2 * MT && MT % 2 == 0 && CA >= 16 && CB >= 16, "whole loads, places of chunks stay in the row");
  __shared__ __attribute__((aligned(16))) char lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  int mt, nt;
  if (!place_tile<4>(blockIdx.x, p.E * mtiles, ntiles, mt, nt)) return;
  const int e = mt / mtiles;
  const int64_t m0 = (int64_t)(mt - e * mtiles) * 16 * MT, n0 = (int64_t)nt * 32 * WN;
  int p0 = 0, n = p.P;
  if (p.offsets) {
    p0 = min(max(p.offsets[e], 0), p.P);
    n = max(min(max(p.offsets[e + 1], 0), p.P) - p0, 0);
  }
  const int last = (n + 63) / 64 - 1;

  // load q of a stage: its rows from (q WN + wave) 64 / C on, chunk by place
  auto at_row = [&](int q, int chunks) { return (q * WN + wave) * (64 / chunks) + lane / chunks; };
  auto col_a = [&](int q) { return ((lane % CA) ^ across_place<false>(at_row(q, CA))) * 16; };
  auto col_b = [&](int q) { return ((lane % CB) ^ across_place<true>(at_row(q, CB))) * 16; };
  const char *const dy = p.dy + p0 * p.lddy + m0 * 2;
  const int64_t x0 = p.perm ? 0 : p0;  // the row that offsets count from
  const char *const xe = p.x + x0 * p.ldx + n0 * 2;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xe, range_of((p.T - x0 - 1) * p.ldx + (p.K - n0) * 2));
  // the entries of the permutation of stage st, asked for a stage ahead and not touched before
  int named[DB];
  auto find_rows = [&](int st) {
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const int row = st * 64 + at_row(q, CB);
      named[q] = row >= n ? -1 : p.perm ? p.perm[p0 + row] : p0 + row;
    }
  };
  auto load = [&](int st, char *to) {
    int at_x[DB];
#pragma unroll
    for (int q = 0; q < DB; ++q) at_x[q] = row_named(p.k_inv, p.T, named[q]);
    find_rows(st + 1);
    asm volatile("" ::: "memory");
    const int64_t d0 = (int64_t)st * 64 * p.lddy;  // the range ends with the expert's rows: past it are zeros
    const __amdgpu_buffer_rsrc_t ry = make_rsrc(dy + d0, range_of((n - st * 64 - 1) * p.lddy + (p.N - m0) * 2));
#pragma unroll
    for (int q = 0; q < DA; ++q)
      load_stage16(ry, to + (q * WN + wave) * 1024, (uint32_t)(at_row(q, CA) * p.lddy) + col_a(q), 0);
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      char *const d = to + BOFF + (q * WN + wave) * 1024;
      if (FAR) load_lds16(at_x[q] >= 0 && n0 * 2 + col_b(q) < p.K * 2 ? xe + at_x[q] * p.ldx + col_b(q) : (const char *)kZeros, d);
      else load_stage16(rx, d, at_x[q] >= 0 ? (uint32_t)((at_x[q] - x0) * p.ldx) + col_b(q) : kNowhere, 0);
    }
    asm volatile("" ::: "memory");
  };
  typename OP::Acc acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = typename OP::Acc{0, 0, 0, 0};

  // the steps, and the order of reads, loads and barriers, of the forward product
  constexpr int S = MT / 2;
  u4 a[2][2], b[2][NT];
  auto read_a = [&](const char *x, int u, int j) {
#pragma unroll
    for (int m = 0; m < 2; ++m) a[(u * S + j) & 1][m] = read_across<false>(x, CA * 16, 0, 2 * j + m, u);
  };
  auto read_b = [&](const char *x, int u) {
#pragma unroll
    for (int i = 0; i < NT; ++i) b[u][i] = read_across<true>(x + BOFF, CB * 16, 4 * wave, i, u);
  };
  find_rows(0);
  if (last >= 0) load(0, lds);
  if (last >= 1) load(1, lds + STAGE);
  wait_vm<0>();
  barrier_keep_loads();
  read_b(lds, 0);
  read_a(lds, 0, 0);
  for (int s = 0; s <= last; ++s) {
    char *const x = lds + (s & 1) * STAGE, *const next = lds + (~s & 1) * STAGE;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (j + 1 < S) read_a(x, u, j + 1);
        else if (u == 0) {
          read_b(x, 1);
          read_a(x, 1, 0);
        } else if (s < last) {
          wait_vm<0>();
          barrier_keep_loads();
          if (s + 2 <= last) load(s + 2, x);
          read_b(next, 0);
          read_a(next, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[i][2 * j + m] = OP::mul(b[u][i], a[(u * S + j) & 1][m], acc[i][2 * j + m]);
        __builtin_amdgcn_sched_barrier(0);
      }
  }

  const bool wide = wide_rows(p.dw_type, p.K);
  const int64_t c = n0 + wave * 32 + 8 * g;
  if (c >= p.K) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = m0 + 16 * m + r;
    if (row >= p.N) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = acc[i / 4][m][i % 4];
    store_values<8>(p.dw, p.dw_type, ((int64_t)e * p.N + row) * p.K + c, p.K - c, wide, v);
  }
}

template <class OP, int WN, int MT, bool FAR>
hipError_t dw(const GroupedDw &p, hipStream_t s) {
  const int64_t mt = (p.N + 16 * MT - 1) / (16 * MT), nt = (p.K + 32 * WN - 1) / (32 * WN);
  hipLaunchKernelGGL((k_grouped_dw<OP, WN, MT, FAR>), dim3((unsigned)((p.E * mt * nt + 7) / 8 * 8)), dim3(64 * WN), 0, s, p, (int)mt, (int)nt);
  return hipGetLastError();
}
template <class OP>
hipError_t choose_dw(const GroupedDw &p, hipStream_t s) {
  if (p.perm && p.T * p.ldx > kRange) return dw<OP, 4, 8, true>(p, s);
  return p.P / p.E > 256 && p.E * p.N * p.K >= (1 << 25) ? dw<OP, 8, 16, false>(p, s) : dw<OP, 4, 8, false>(p, s);
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

hipError_t launch_grouped_dw(const GroupedDw &p, hipStream_t s) { return p.type == DS4MOE_BF16 ? choose_dw<OpBf16>(p, s) : choose_dw<OpF16>(p, s); }

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
