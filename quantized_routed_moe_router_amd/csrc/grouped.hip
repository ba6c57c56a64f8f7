// Products grouped by expert, y[p] = W_e x[row(p)], of bf16, fp16 or 8-bit
// integer operands; the dense product of 8-bit integers, which is one group of
// all rows; and the gradient of the rows, dx[p] = W_e^T dy[p], which is the
// same product of weights that lie across.
//
// A workgroup of WN waves has up to 256 rows of one expert and 32 WN columns
// of y, 32 a wave.  Both operands are staged in LDS, 128 bytes of a row (64 or
// 128 terms of the sums) at a time, by loads that bypass the registers.
// Weights are the matrix instructions' rows and activations their columns: row
// 4 g + v of a wave's i-th group of 16 is column 8 g + 4 i + v of it, so that a
// lane's results are 8 adjacent columns of one row of y.
//
// What bounds it.  Many rows an expert: no one unit.  16384 rows of 8 experts,
// 2048 x 4096 bf16, take 264 us (1.04 PFLOP/s).  The matrix units are busy for
// 49 % of the cycles, at 1.85 GHz; a SIMD holds 1.8 of its two waves on average,
// the last round of tiles not being full, and the waves stand at waits and
// barriers for 38 % of their time.  One dense 8192^3 runs at 1.39 PFLOP/s (the
// library's at 1.54) with the units busy for 66 %, and a loop of nothing but
// matrix instructions for 86 %.  Few rows: reading the weights, 256 experts'
// 4.3 GB for 64 rows each in 800 us (5.5 TB/s), the 1.6 GB of the 8-bit experts
// that have rows of a skewed choice in 324.  The dense 8-bit product of 2048
// rows, 4096 x 4096, one round of 512 tiles of 32 stages, takes 36.7 to 39.5 us
// (1.74 to 1.87 POP/s, units busy for 40 % at 1.9 GHz; the library's, without
// scales, 40.1).  Left out, of 8192^3 in 784 us: matrix instructions of 32 x 32
// 862, stages of 64 bytes 850, buffers handed on in parts 787, row tiles in
// groups of 2, 8 or 16 by all columns 817, 791, 855.  Not built: workgroups that
// load their next tile under the results of this one.
#include "grouped_dev.h"

namespace ds4 {

namespace {

constexpr int LDS_PER_WAVE = 20 << 10;

// One workgroup's tile: rows t (up to 16 MT), columns n0 .. of its expert, in
// NB buffers of stages.  FAR: rows of x that 32-bit offsets do not reach.
template <class OP, bool TURNED, int WN, int MT, int NB, bool FAR>
__device__ __forceinline__ void multiply_tile(const Grouped &p, const Segment &t, int64_t n0, char *lds) {
  constexpr int NT = 2, DA = (2 * MT + WN - 1) / WN, DB = 4;  // groups of 16 weight rows; loads of 8 rows per wave
  constexpr int BOFF = DA * WN * 1024, STAGE = BOFF + DB * WN * 1024;
  static_assert(NB * STAGE <= WN * LDS_PER_WAVE, "the buffers fit");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  const int last = (int)((p.Kb + 127) / 128) - 1, edge = (int)(p.Kb - (int64_t)last * 128) / 16;  // chunks of the last stage

  // The lane's source of load q: row 8 (q WN + wave) + lane / 8, its chunk by
  // the place that lane l's bytes get.  Rows past the end, and rows that the
  // permutation does not name, are zeros.
  const char *const we = p.w + (TURNED ? (int64_t)t.e * p.N * p.Kb + n0 * 2 : ((int64_t)t.e * p.N + n0) * p.Kb);
  const int64_t wbytes = TURNED ? p.N * p.Kb - n0 * 2 : (p.N - n0) * p.Kb;  // to the matrix' end
  const int64_t x0 = p.perm ? 0 : t.p0;  // the row that offsets count from
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + x0 * p.ldx, range_of((p.T - x0 - 1) * p.ldx + p.Kb));
  auto row = [&](int q) { return (q * WN + wave) * 8 + (lane >> 3); };
  auto chunk_a = [&](int q) { return (lane & 7) ^ place8(row(q) & 15); };
  auto chunk_b = [&](int q) { return (lane & 7) ^ place8((row(q) >> 3 & 3) << 2 | (row(q) & 3)); };
  constexpr int CW = 4 * WN;  // chunks of a row of turned weights
  auto turned_row = [&](int q) { return (q * WN + wave) * (64 / CW) + lane / CW; };
  uint32_t sa[DA], sb[DB];
  int at_x[DA];
#pragma unroll
  for (int q = 0; q < DA; ++q) {
    at_x[q] = row(q) < t.n ? row_of(p.perm, p.k_inv, p.T, t.p0 + row(q)) : -1;
    sa[q] = at_x[q] < 0 ? kNowhere : (uint32_t)((at_x[q] - x0) * p.ldx) + chunk_a(q) * 16;
  }
#pragma unroll
  for (int q = 0; q < DB; ++q)
    sb[q] = TURNED ? (uint32_t)(turned_row(q) * p.N * 2) + ((lane % CW) ^ across_place<true>(turned_row(q))) * 16
                   : (uint32_t)(row(q) * p.Kb) + chunk_b(q) * 16;
  auto load = [&](int st, char *to) {
    const bool whole = st < last || edge == 8;
#pragma unroll
    for (int q = 0; q < DA; ++q) {
      char *const d = to + (q * WN + wave) * 1024;
      const bool in = whole || chunk_a(q) < edge;
      if (FAR) load_lds16(in && at_x[q] >= 0 ? p.x + at_x[q] * p.ldx + chunk_a(q) * 16 + (int64_t)st * 128 : (const char *)kZeros, d);
      else load_stage16(rx, d, in ? sa[q] : kNowhere, st * 128);
    }
    // turned, a stage is 64 rows, and the range ends with the matrix
    const int64_t w0 = TURNED ? st * 128 * p.N : 0;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(we + w0, range_of(wbytes - w0));
#pragma unroll
    for (int q = 0; q < DB; ++q)
      load_stage16(rw, to + BOFF + (q * WN + wave) * 1024, TURNED || whole || chunk_b(q) < edge ? sb[q] : kNowhere, TURNED ? 0 : st * 128);
    asm volatile("" ::: "memory");
  };
  typename OP::Acc acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = typename OP::Acc{0, 0, 0, 0};

  // The products of 64 bytes of the rows go in steps of two groups of rows.  A
  // step's fragments are read under the step before it, those of the next
  // stage's first step under this one's last, behind a barrier that says that
  // the next stage has landed and that this one has been read; the buffer that
  // it frees is filled again at once.
  constexpr int S = (MT + 1) / 2;
  const int fa = r * 128, fb = BOFF + (wave * 32 + 8 * (r >> 2) + (r & 3)) * 128, f0 = (g ^ place8(r)) * 16;
  const uint32_t tb = BOFF + across_at<true>(64 * WN, 4 * wave, 0);
  u4 a[2][2], b[2][NT];
  auto read_a = [&](const char *x, int u, int j) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
      if (2 * j + m < MT) a[(u * S + j) & 1][m] = *reinterpret_cast<const u4 *>(x + fa + (2 * j + m) * 2048 + (f0 ^ 64 * u));
  };
  auto read_b = [&](const char *x, int u) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
      b[u][i] = TURNED ? read_across((lds_at)x + tb + (32 * 64 * WN * u + 8 * i), 64 * WN) : *reinterpret_cast<const u4 *>(x + fb + i * 512 + (f0 ^ 64 * u));
  };
#pragma unroll
  for (int i = 0; i < NB; ++i)
    if (i <= last) load(i, lds + i * STAGE);
  if (last >= NB - 1) wait_vm<(NB - 1) * (DA + DB)>();
  else wait_vm<0>();
  barrier_keep_loads();
  char *x = lds;
  read_b(x, 0);
  read_a(x, 0, 0);
  for (int s = 0; s <= last; ++s) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (j + 1 < S) read_a(x, u, j + 1);
        else if (u == 0) {
          read_b(x, 1);
          read_a(x, 1, 0);
        } else if (s < last) {
          if (s + NB - 1 <= last) wait_vm<(NB - 2) * (DA + DB)>();
          else wait_vm<0>();
          barrier_keep_loads();
          if (s + NB <= last) load(s + NB, x);
          x = x + STAGE == lds + NB * STAGE ? lds : x + STAGE;
          read_b(x, 0);
          read_a(x, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i)
            if (2 * j + m < MT) acc[i][2 * j + m] = OP::mul(b[u][i], a[(u * S + j) & 1][m], acc[i][2 * j + m]);
        __builtin_amdgcn_sched_barrier(0);
      }
  }

  const bool wide = wide_rows(p.y_type, p.ldy);
  const int64_t n_wave = n0 + wave * 32, n = n_wave + 8 * g;
  if (!wide) barrier_keep_loads();  // the buffers have been read
  if (n_wave >= p.N) return;
  float sw[8];
  if (OP::SCALED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sw[i] = p.ws[(int64_t)t.e * p.N + min(n + i, p.N - 1)];
  }
  float *const own = reinterpret_cast<float *>(lds + wave * 16 * 36 * 4);  // 16 rows of 32 values, 4 apart
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int at_row = 16 * m + r;
    float sx = 1.0f;
    if (OP::SCALED) {
      const int at = at_row < t.n ? row_of(p.perm, p.k_inv, p.T, t.p0 + at_row) : -1;
      sx = at < 0 ? 0.0f : p.xs[at];
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = OP::SCALED ? (float)acc[i / 4][m][i % 4] * sx * sw[i] : (float)acc[i / 4][m][i % 4];
    if (wide) {
      if (at_row < t.n && n < p.N) store_values<8>(p.y, p.y_type, (int64_t)(t.p0 + at_row) * p.ldy + n, p.N - n, true, v);
      continue;
    }
    // Rows that begin anywhere: eight values of 16 rows each would go out one
    // by one from 64 places.  Through LDS two whole rows of 32 go at a time.
    *reinterpret_cast<f4 *>(own + r * 36 + 8 * g) = f4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f4 *>(own + r * 36 + 8 * g + 4) = f4{v[4], v[5], v[6], v[7]};
    lds_order();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 2 * i + (lane >> 5), c = lane & 31;
      const float u[1] = {own[row * 36 + c]};
      if (16 * m + row < t.n && n_wave + c < p.N) store_values<1>(p.y, p.y_type, (int64_t)(t.p0 + 16 * m + row) * p.ldy + n_wave + c, 1, false, u);
    }
    lds_order();
  }
}

// Eight waves (256 columns) with the LDS of a CU, or four (128 columns) with
// half of it.  HEIGHT: of the tiles, 0 for one that suits the numbers of rows;
// a tile runs in the smallest instance that has its rows.
template <class OP, bool TURNED, int WN, int HEIGHT>
__global__ __launch_bounds__(64 * WN, 2) void k_grouped(Grouped p, int ntiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  if (TURNED)
    for (int64_t i = (int64_t)blockIdx.x * (64 * WN) + threadIdx.x; i < p.n_places; i += (int64_t)gridDim.x * (64 * WN)) p.places[i] = -1;
  Finder f;
  f.load(p.offsets, p.E, p.P);
  if (HEIGHT) f.set_height(HEIGHT);
  else if (WN == 8) f.choose_height<8>({256, 224, 192, 160, 128}, ntiles);
  else f.choose_height<9>({192, 160, 128, 64}, ntiles);
  const int mtiles = f.count();
  int mt, nt;
  if (!place_tile<4>(blockIdx.x, mtiles, ntiles, mt, nt)) return;
  const Segment t = f.find(mt);
  const int64_t n0 = (int64_t)nt * 32 * WN;
  if (t.e < 0) {
    zero_rows(p.y, p.y_type, p.ldy, t.p0, t.n, n0, min(n0 + 32 * WN, p.N));
    return;
  }
  if (HEIGHT == 64 || t.n <= 64) return multiply_tile<OP, TURNED, WN, 4, WN == 8 ? 4 : 3, false>(p, t, n0, lds);
  if constexpr (HEIGHT != 64) {
    if (HEIGHT == 128 || t.n <= 128) return multiply_tile<OP, TURNED, WN, 8, WN == 8 ? 3 : 2, false>(p, t, n0, lds);
  }
  if constexpr (HEIGHT == 0) {
    if (t.n <= 160) return multiply_tile<OP, TURNED, WN, 10, 2, false>(p, t, n0, lds);
    if (WN == 4 || t.n <= 192) return multiply_tile<OP, TURNED, WN, 12, 2, false>(p, t, n0, lds);
    if constexpr (WN == 8) {
      if (t.n <= 224) return multiply_tile<OP, TURNED, WN, 14, 2, false>(p, t, n0, lds);
      multiply_tile<OP, TURNED, WN, 16, 2, false>(p, t, n0, lds);
    }
  }
}
template <class OP>
__global__ __launch_bounds__(512, 2) void k_grouped_far(Grouped p, int ntiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  Finder f;
  f.load(p.offsets, p.E, p.P);
  f.set_height(128);
  const int mtiles = f.count();
  int mt, nt;
  if (!place_tile<4>(blockIdx.x, mtiles, ntiles, mt, nt)) return;
  const Segment t = f.find(mt);
  const int64_t n0 = (int64_t)nt * 256;
  if (t.e < 0) zero_rows(p.y, p.y_type, p.ldy, t.p0, t.n, n0, min(n0 + 256, p.N));
  else multiply_tile<OP, false, 8, 8, 3, true>(p, t, n0, lds);
}

template <class OP, bool TURNED, int WN, int HEIGHT>
hipError_t tiled(const Grouped &p, hipStream_t s) {
  constexpr GroupedForm f{WN, HEIGHT};
  const dim3 g((unsigned)grouped_workgroups(f, p.offsets, p.E, p.P, p.N));
  hipLaunchKernelGGL((k_grouped<OP, TURNED, WN, HEIGHT>), g, dim3(64 * WN), WN * LDS_PER_WAVE, s, p, (int)grouped_col_tiles(f, p.N));
  return hipGetLastError();
}
template <class OP>
hipError_t tiled_far(const Grouped &p, hipStream_t s) {
  constexpr GroupedForm f{8, 128};
  const dim3 g((unsigned)grouped_workgroups(f, p.offsets, p.E, p.P, p.N));
  hipLaunchKernelGGL(k_grouped_far<OP>, g, dim3(512), 8 * LDS_PER_WAVE, s, p, (int)grouped_col_tiles(f, p.N));
  return hipGetLastError();
}

template <class OP>
hipError_t choose(const Grouped &p, hipStream_t s) {
  const GroupedForm f = grouped_form(p.offsets, p.E, p.P, p.N);
  if (f.waves == 8) return f.height ? tiled<OP, false, 8, 128>(p, s) : tiled<OP, false, 8, 0>(p, s);
  return f.height ? tiled<OP, false, 4, 64>(p, s) : tiled<OP, false, 4, 0>(p, s);
}
template <class OP>
hipError_t choose_turned(const Grouped &p, hipStream_t s) {
  const GroupedForm f = grouped_turned_form(p.E, p.P, p.N);
  if (f.waves == 8) return tiled<OP, true, 8, 128>(p, s);
  return f.height ? tiled<OP, true, 4, 64>(p, s) : tiled<OP, true, 4, 0>(p, s);
}

}  // namespace

hipError_t launch_grouped(const Grouped &p, hipStream_t s) {
  if (p.turned) return p.type == DS4MOE_BF16 ? choose_turned<OpBf16>(p, s) : choose_turned<OpF16>(p, s);
  if (grouped_is_few(p.offsets, p.E, p.P)) return launch_grouped_few(p, s);
  if (p.perm && p.T * p.ldx > kRange)  // rows that 32-bit offsets do not reach
    return p.type == DS4MOE_BF16 ? tiled_far<OpBf16>(p, s) : p.type == DS4MOE_F16 ? tiled_far<OpF16>(p, s) : tiled_far<OpI8>(p, s);
  if (p.type == DS4MOE_BF16) return choose<OpBf16>(p, s);
  if (p.type == DS4MOE_F16) return choose<OpF16>(p, s);
  return choose<OpI8>(p, s);
}

}  // namespace ds4
