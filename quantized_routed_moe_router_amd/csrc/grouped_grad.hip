// Gradients of the products grouped by expert: of the weights,
//   dW_e = sum over p of dy[p] x[row(p)]^T,
// in bf16 or fp16 operands, and the sum of the gradients of rows that several
// experts share.  (The gradient of the rows is a product by turned weights.)
//
// A workgroup of 2 WN waves has 32 MT rows and 64 WN columns of one dW_e, 32
// terms of the sum at a time.  Both operands lie across.
//
// With many rows an expert no one unit bounds it: 8 experts of 1024 rows, 2048
// x 4096, 151 us (0.91 PFLOP/s; the library's product of these sizes reaches
// 1.5), the matrix units busy for 39 % of the cycles at 2.1 GHz, the waves at
// waits and barriers for 35 % of their time; a workgroup's first loads and its
// results are not under another's products.  With few rows it is writing dW: 256 experts of 64 rows,
// 1170 us for 4.4 GB (3.7 TB/s).  Left out, of 8192 rows: tiles of 128 x 256
// 151 us and 1315 with 64 rows an expert; 256 x 256 in two buffers 148 and
// 1237; one workgroup a CU that goes round 157 and 1298.
#include "grouped_dev.h"

namespace ds4 {

namespace {

// PERM: rows by a permutation.  FAR: rows that 32-bit offsets do not reach.
template <class OP, int WN, int MT, int NB, bool PERM, bool FAR>
__global__ __launch_bounds__(128 * WN, 2) void k_grouped_dw(GroupedDw p, int mtiles, int ntiles) {
  constexpr int WAVES = 2 * WN, NT = 4, BM = 32 * MT, BN = 64 * WN;
  constexpr int CA = BM / 8, CB = BN / 8;                        // chunks of a staged row
  constexpr int DA = CA / 2 / WAVES, DB = CB / 2 / WAVES, D = DA + DB;  // loads per wave
  constexpr int BOFF = BM * 64, STAGE = BOFF + BN * 64;
  static_assert(DA * WAVES * 2 == CA && CA == CB && MT % 4 == 0 && CA >= 16 && NB % 2 == 0,
                "whole loads, places of chunks stay in the row, load q has the same rows of both operands");
  __shared__ __attribute__((aligned(16))) char lds[NB * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  int mt, nt;
  if (!place_tile<4>(blockIdx.x, p.E * mtiles, ntiles, mt, nt)) return;
  const int e = mt / mtiles;
  const int64_t m0 = (int64_t)(mt - e * mtiles) * BM, n0 = (int64_t)nt * BN;
  int p0 = 0, n = p.P;
  if (p.offsets) {
    p0 = min(max(p.offsets[e], 0), p.P);
    n = max(min(max(p.offsets[e + 1], 0), p.P) - p0, 0);
  }
  const int last = (n + 31) / 32 - 1;

  // Load q of a stage: its rows from (q WAVES + wave) 64 / C on, chunk by place.
  // The ranges of dy, and of x in order, end with the expert's rows: past them
  // are zeros.
  auto row_a = [&](int q) { return (q * WAVES + wave) * (64 / CA) + lane / CA; };
  auto row_b = [&](int q) { return (q * WAVES + wave) * (64 / CB) + lane / CB; };
  auto col_a = [&](int q) { return ((lane % CA) ^ across_place<false>(row_a(q))) * 16; };
  auto col_b = [&](int q) { return ((lane % CB) ^ across_place<true>(row_b(q))) * 16; };
  const uint32_t lddy = (uint32_t)p.lddy, ldx = (uint32_t)p.ldx;
  const char *const dy = p.dy + p0 * p.lddy + m0 * 2;
  const char *const xe = p.x + (PERM ? 0 : p0 * p.ldx) + n0 * 2;
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(dy, range_of((int64_t)(n - 1) * p.lddy + (p.N - m0) * 2));
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(xe, range_of((int64_t)((PERM ? p.T : min(n, p.T - p0)) - 1) * p.ldx + (p.K - n0) * 2));
  uint32_t sa[DA], sb[DB];
#pragma unroll
  for (int q = 0; q < DA; ++q) sa[q] = row_a(q) * lddy + col_a(q);
#pragma unroll
  for (int q = 0; q < DB; ++q) sb[q] = PERM ? 0 : row_b(q) * ldx + col_b(q);
  // The permutation's entries of a stage are asked for two stages before they
  // are turned into offsets, and that is done in the middle of the stage whose
  // end issues the loads: behind the barrier, where all waves are at the same
  // place, nothing is left to work out.
  int named[2][DB];
  auto ask = [&](int st, int (&to)[DB]) {
#pragma unroll
    for (int q = 0; q < DB; ++q) to[q] = p.perm[p0 + min(st * 32 + row_b(q), n - 1)];
  };
  // A position that names no row has zeros of dy too: what stands there, a NaN
  // or an infinity, adds nothing.
  int at_x[DB];
  uint32_t named_a[DA];
  auto prepare = [&](int st, const int (&from)[DB]) {
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const int at = row_named(p.k_inv, p.T, from[q]);
      at_x[q] = st * 32 + row_b(q) < n ? at : -1;
      sb[q] = at_x[q] >= 0 ? at * ldx + col_b(q) : kNowhere;
      named_a[q] = at_x[q] >= 0 ? sa[q] : kNowhere;
    }
  };
  auto load = [&](int st, char *to) {
#pragma unroll
    for (int q = 0; q < DA; ++q) {
      char *const d = to + (q * WAVES + wave) * 1024;
      if (FAR) load_lds16((PERM ? at_x[q] >= 0 : st * 32 + row_a(q) < n) && m0 * 2 + col_a(q) < p.N * 2 ? dy + (int64_t)(st * 32 + row_a(q)) * p.lddy + col_a(q) : (const char *)kZeros, d);
      else load_stage16(ry, d, PERM ? named_a[q] : sa[q], st * 32 * lddy);
    }
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      char *const d = to + BOFF + (q * WAVES + wave) * 1024;
      if (FAR) {
        const int64_t at = PERM ? at_x[q] : st * 32 + row_b(q) < min(n, p.T - p0) ? st * 32 + row_b(q) : -1;
        load_lds16(at >= 0 && n0 * 2 + col_b(q) < p.K * 2 ? xe + at * p.ldx + col_b(q) : (const char *)kZeros, d);
      } else load_stage16(rx, d, sb[q], PERM ? 0 : st * 32 * ldx);
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
  uint32_t la[MT], lb[NT / 2];
#pragma unroll
  for (int m = 0; m < MT; ++m) la[m] = across_at<false>(CA * 16, 2 * MT * wm, m);
#pragma unroll
  for (int i = 0; i < NT / 2; ++i) lb[i] = BOFF + across_at<true>(CB * 16, 8 * wn, 2 * i);
  u4 a[2][2], b[2][NT];
  auto read_a = [&](const char *x, int u, int j) {
#pragma unroll
    for (int m = 0; m < 2; ++m) a[(u * S + j) & 1][m] = read_across((lds_at)x + la[2 * j + m], CA * 16);
  };
  auto read_b = [&](const char *x, int u) {
#pragma unroll
    for (int i = 0; i < NT; ++i) b[u][i] = read_across((lds_at)x + lb[i / 2] + 8 * (i & 1), CB * 16);
  };
  char *x = lds;
  int s = 0;
  bool more = last >= 0;
  // `all`: the sum has stages for all that is asked for here
  auto begin = [&](bool all) __attribute__((always_inline)) {
    int first[NB][DB];
    if (PERM) {
#pragma unroll
      for (int i = 0; i < NB; ++i) ask(i, first[i]);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (PERM) {
        if (i >= NB - 2) ask(i + 2, named[i - (NB - 2)]);  // in the order of the loop, whose waits count them
        prepare(i, first[i]);
      }
      if (all || i <= last) load(i, lds + i * STAGE);
    }
  };
  auto start = [&](bool all) __attribute__((always_inline)) {
    // younger than the first stage's loads: those of NB - 1 stages, and of the entries that are asked for behind it
    // (not counted where nobody may need them: they might not be asked for)
    if (all) wait_vm<(NB - 1) * D + (PERM ? (NB > 2 ? 2 : 1) * DB : 0)>();
    else if (last >= NB - 1) wait_vm<(NB - 1) * D>();
    else wait_vm<0>();
    barrier_keep_loads();
    read_b(x, 0);
    read_a(x, 0, 0);
  };
  // `all`: NB more stages follow this one
  auto stage = [&](bool all, int u) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if (PERM && j == S / 2 && (all || s + NB <= last)) {
        prepare(s + NB, named[u]);
        ask(s + NB + 2, named[u]);
        asm volatile("" ::: "memory");
      }
      if (j + 1 < S) read_a(x, u, j + 1);
      else if (all || s < last) {
        // younger than the next stage's loads: those of NB - 2 stages and the entries asked for in NB - 1 (counted as above)
        if (all) wait_vm<(NB - 2) * D + (PERM ? (NB - 1) * DB : 0)>();
        else if (s + NB - 1 <= last) wait_vm<(NB - 2) * D>();
        else wait_vm<0>();
        barrier_keep_loads();
        if (all || s + NB <= last) load(s + NB, x);
        x = x + STAGE == lds + NB * STAGE ? lds : x + STAGE;
        read_b(x, u ^ 1);
        read_a(x, u ^ 1, 0);
        ++s;
      } else more = false;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][2 * j + m] = OP::mul(b[u][i], a[(u * S + j) & 1][m], acc[i][2 * j + m]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Stages whose loads depend on nothing have a loop of their own: there the
  // compiler knows how many loads are younger than an entry that it waits for.
  // Behind a condition it waits for all of them.
  if (last > NB) {
    begin(true);
    start(true);
    while (s + NB < last) {
      stage(true, 0);
      stage(true, 1);
    }
  } else {
    if (more) begin(false);
    start(false);
  }
  while (more) {
    stage(false, 0);
    if (more) stage(false, 1);
  }

  const bool wide = wide_rows(p.dw_type, p.K);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = m0 + wm * 16 * MT + 16 * m + r;
    if (row >= p.N) continue;
#pragma unroll
    for (int i = 0; i < NT; i += 2) {
      const int64_t c = n0 + wn * 64 + 16 * i + 8 * g;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[i + j / 4][m][j % 4];
      if (c < p.K) store_values<8>(p.dw, p.dw_type, ((int64_t)e * p.N + row) * p.K + c, p.K - c, wide, v);
    }
  }
}

template <class OP, int WN, int MT, int NB, bool FAR>
hipError_t dw(const GroupedDw &p, hipStream_t s) {
  static_assert(32 * MT == 64 * WN, "square tiles");
  const int64_t mt = (p.N + 32 * MT - 1) / (32 * MT), nt = (p.K + 64 * WN - 1) / (64 * WN);
  const dim3 g((unsigned)grouped_dw_workgroups(WN == 4, p.E, p.N, p.K)), b(128 * WN);
  if (p.perm) hipLaunchKernelGGL((k_grouped_dw<OP, WN, MT, NB, true, FAR>), g, b, 0, s, p, (int)mt, (int)nt);
  else hipLaunchKernelGGL((k_grouped_dw<OP, WN, MT, NB, false, FAR>), g, b, 0, s, p, (int)mt, (int)nt);
  return hipGetLastError();
}
template <class OP>
hipError_t choose_dw(const GroupedDw &p, hipStream_t s) {
  // offsets of an expert's rows, up to 31 past the last in the last stage, and of those that the permutation names
  const int64_t end = (int64_t)p.P + 31;
  if (end * p.lddy > kRange || (p.perm ? p.T : end) * p.ldx > kRange) return dw<OP, 2, 4, 2, true>(p, s);
  return grouped_dw_large(p.E, p.N, p.K) ? dw<OP, 4, 8, 4, false>(p, s) : dw<OP, 2, 4, 2, false>(p, s);
}

// ---------------------------------------------------------------- gradients of shared rows
__global__ __launch_bounds__(256) void k_grouped_no_places(int32_t *places, int A) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < A) places[i] = -1;
}

// The positions that have an expert.
__device__ __forceinline__ int begin_of(const GroupedPlaces &q) { return min(max(q.offsets[0], 0), q.P); }
__device__ __forceinline__ int end_of(const GroupedPlaces &q) { return max(begin_of(q), min(max(q.offsets[q.E], 0), q.P)); }

// An assignment's place is one of its positions (-1: none); next[position] is
// another, and so on: a list in no particular order, which nearly always has
// one.  kMore in the place says that it has more: whoever comes to a place that
// is taken sets it behind its own entry.  Positions without an expert are in
// none.
constexpr int kMore = 1 << 30;  // positions are below 2^23
__global__ __launch_bounds__(256) void k_grouped_places(GroupedPlaces q) {
  const int i = blockIdx.x * 256 + threadIdx.x, a = i < q.P ? q.perm[i] : -1;
  if (i < begin_of(q) || i >= end_of(q) || a < 0 || a >= q.A) return;
  const int before = atomicExch(q.place + a, i);
  q.next[i] = before < 0 ? -1 : before & (kMore - 1);
  if (before >= 0) atomicOr(q.place + a, kMore);
}

// dx[t] = sum over j of the rows of its assignments, in the order of j and of
// the positions of each, in fp32 with one rounding.  The rows are fp32 so that
// there is one.  Bound by the memory: two rows each of 4096 tokens, 4096 wide,
// 29 us (134 MB in, 34 out, 5.8 TB/s).
//
// Where an assignment stands several times, its list is put in order first.  Up
// to LIST positions are sorted in LDS; an assignment of more is looked for in
// the permutation from end to end, which has at most P / LIST of these.  Two
// positions each of 65536 tokens, 512 wide, as tokens' numbers: the gradient of
// the rows in 201 us, 190 by assignments that are distinct.
template <int NV>
__global__ __launch_bounds__(256) void k_grouped_add_up(void *dx, int64_t ldo, int o_type, const float *rows, GroupedPlaces q, int T, int k, int64_t K) {
  constexpr int LIST = 256;
  __shared__ int list[LIST], sorted[LIST], length;
  __shared__ uint64_t found[4];
  const int tid = threadIdx.x;
  const int threads = blockDim.x;  // no more waves than columns give work to
  const int64_t c = ((int64_t)blockIdx.y * threads + tid) * NV;
  const bool in = c < K;
  float v[NV];
  auto add = [&](int at) {
    if (!in) return;
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const f4 u = *reinterpret_cast<const f4 *>(rows + at * K + c + i);
#pragma unroll
      for (int l = 0; l < 4; ++l) v[i + l] += u[l];
    }
  };
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.0f;
  };
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    clear();
    int more = 0;
    for (int j = 0; j < k; ++j) {
      const int at = q.place[t * k + j];
      if (at < 0) continue;
      more |= at & kMore;
      add(at & (kMore - 1));
    }
    if (more) {
      clear();
      for (int j = 0; j < k; ++j) {
        const int a = (int)(t * k + j), head = q.place[a];
        if (head < 0) continue;
        __syncthreads();  // what was in LDS has been read
        if (tid == 0) {
          int n = 0, at = head & (kMore - 1);
          for (; at >= 0 && n < LIST; at = q.next[at]) list[n++] = at;
          length = at >= 0 ? -1 : n;
        }
        __syncthreads();
        const int n = length;
        for (int l = tid; l < n; l += threads) {
          int rank = 0;
          for (int i = 0; i < n; ++i) rank += list[i] < list[l];
          sorted[rank] = list[l];
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) add(sorted[i]);
        if (n >= 0) continue;
        for (int from = begin_of(q), end = end_of(q); from < end; from += threads) {
          const uint64_t here = __ballot(from + tid < end && q.perm[min(from + tid, q.P - 1)] == a);
          if ((tid & 63) == 0) found[tid >> 6] = here;
          __syncthreads();
          for (int w = 0; w < threads / 64; ++w)
            for (uint64_t m = found[w]; m; m &= m - 1) add(from + 64 * w + __ffsll((unsigned long long)m) - 1);
          __syncthreads();
        }
      }
    }
    if (in) store_values<NV>(dx, o_type, t * ldo + c, K - c, wide_rows(o_type, ldo), v);
  }
}

}  // namespace

hipError_t launch_grouped_dw(const GroupedDw &p, hipStream_t s) { return p.type == DS4MOE_BF16 ? choose_dw<OpBf16>(p, s) : choose_dw<OpF16>(p, s); }

hipError_t launch_grouped_places(const GroupedPlaces &q, hipStream_t s) {
  if (q.P) hipLaunchKernelGGL(k_grouped_places, dim3((q.P + 255) / 256), dim3(256), 0, s, q);
  else hipLaunchKernelGGL(k_grouped_no_places, dim3((q.A + 255) / 256), dim3(256), 0, s, q.place, q.A);
  return hipGetLastError();
}

hipError_t launch_grouped_add_up(void *dx, int64_t ldo, int32_t o_type, const float *rows, const GroupedPlaces &q, int32_t T, int32_t k,
                                 int64_t K, hipStream_t s) {
  const unsigned threads = K < 2048 ? (unsigned)((K + 511) / 512 * 64) : 256;
  hipLaunchKernelGGL(k_grouped_add_up<8>, dim3((unsigned)(T < (1 << 20) ? T : 1 << 20), (unsigned)((K + 2047) / 2048)), dim3(threads), 0, s, dx, ldo,
                     o_type, rows, q, T, k, K);
  return hipGetLastError();
}

}  // namespace ds4
