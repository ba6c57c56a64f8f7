// Products grouped by expert, y[p] = W_e x[row(p)], of bf16, fp16 or 8-bit
// integer operands, and the dense product of 8-bit integers, which is one
// group of all rows.
//
// A workgroup has BM rows of one expert and BN of its weight rows.  Both are
// staged in LDS, 128 bytes of a row (64 or 128 columns) at a time, by loads
// that bypass the registers, NB buffers deep; WM x WN waves share the tile.
// Weights are the matrix instructions' rows and activations their columns:
// row 4 g + v of a wave's i-th group of 16 is weight row 4 NT g + 4 i + v of
// it, so that a lane's results are 4 NT adjacent columns of one row of y.
#include "grouped_dev.h"

namespace ds4 {

namespace {

template <class OP, int BM, int BN, int WM, int WN, int NB>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_grouped(Grouped p, int ntiles) {
  constexpr int WAVES = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int STAGE = (BM + BN) * 128, DA = BM / 8 / WAVES, DB = BN / 8 / WAVES;  // loads of 8 rows per wave
  static_assert(DA * 8 * WAVES == BM && DB * 8 * WAVES == BN && BN / WN % 64 == 0, "whole loads, whole groups");
  __shared__ __attribute__((aligned(16))) char lds[NB * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  Finder<BM> f;
  const int mtiles = f.count(p.offsets, p.E, p.P);
  int mt, nt;
  if (!place_tile<4>(blockIdx.x, mtiles, ntiles, mt, nt)) return;
  const Segment t = f.find(mt);
  const int64_t n0 = (int64_t)nt * BN;
  if (t.e < 0) {
    zero_rows(p.y, p.y_type, p.ldy, t.p0, t.n, n0, min(n0 + BN, p.N));
    return;
  }
  const char *const zeros = (const char *)kZeros;
  const int last = (int)((p.Kb + 127) / 128) - 1, edge = (int)(p.Kb - (int64_t)last * 128) / 16;  // chunks of the last stage

  // The lane's source of load q: row 8 (q WAVES + wave) + lane / 8, its chunk
  // by the place that lane l's bytes get.  Rows past the end repeat the last
  // one (their results are not stored).
  const char *sa[DA], *sb[DB];
  int step[DA], ca[DA], cb[DB];
#pragma unroll
  for (int q = 0; q < DA; ++q) {
    const int row = (q * WAVES + wave) * 8 + (lane >> 3);
    const int at = row_of(p.perm, p.k_inv, p.T, p.k, t.p0 + min(row, t.n - 1));
    ca[q] = (lane & 7) ^ place8(row & 15);
    step[q] = at < 0 ? 0 : 128;
    sa[q] = at < 0 ? zeros : p.x + at * p.ldx + ca[q] * 16;
  }
  const char *const we = p.w + (int64_t)t.e * p.N * p.Kb;
#pragma unroll
  for (int q = 0; q < DB; ++q) {
    const int row = (q * WAVES + wave) * 8 + (lane >> 3), in = row % (16 * NT);
    cb[q] = (lane & 7) ^ place8((in / (4 * NT)) << 2 | (in & 3));
    sb[q] = we + min(n0 + row, p.N - 1) * p.Kb + cb[q] * 16;
  }
  auto load = [&](int st, char *to) {
    const bool short_ = st == last && edge < 8;
#pragma unroll
    for (int q = 0; q < DA; ++q) {
      const char *s = sa[q] + (int64_t)st * step[q];
      if (short_ && ca[q] >= edge) s = zeros;
      load_lds16(s, to + (q * WAVES + wave) * 1024);
    }
#pragma unroll
    for (int q = 0; q < DB; ++q) {
      const char *s = sb[q] + (int64_t)st * 128;
      if (short_ && cb[q] >= edge) s = zeros;
      load_lds16(s, to + BM * 128 + (q * WAVES + wave) * 1024);
    }
    asm volatile("" ::: "memory");
  };
  typename OP::Acc acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = typename OP::Acc{0, 0, 0, 0};

  const int fa = (wm * 16 * MT + r) * 128, fb = BM * 128 + (wn * 16 * NT + 4 * NT * (r >> 2) + (r & 3)) * 128;
  const int f0 = (g ^ place8(r)) * 16;
#pragma unroll
  for (int i = 0; i < NB - 1; ++i)
    if (i <= last) load(i, lds + i * STAGE);
  if (last >= NB - 2) wait_vm<(NB - 2) * (DA + DB)>();
  else wait_vm<0>();
  barrier_keep_loads();
  const char *x = lds;
  char *in = lds + (NB - 1) * STAGE;
  for (int s = 0; s <= last; ++s) {
    if (s + NB - 1 <= last) load(s + NB - 1, in);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u4 a[MT], b[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) b[i] = *reinterpret_cast<const u4 *>(x + fb + i * 512 + (f0 ^ 64 * h));
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m] = *reinterpret_cast<const u4 *>(x + fa + m * 2048 + (f0 ^ 64 * h));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][m] = OP::mul(b[i], a[m], acc[i][m]);
    }
    if (s + NB - 1 <= last) wait_vm<(NB - 2) * (DA + DB)>();
    else wait_vm<0>();
    barrier_keep_loads();
    x = x + STAGE == lds + NB * STAGE ? lds : x + STAGE;
    in = in + STAGE == lds + NB * STAGE ? lds : in + STAGE;
  }

  const bool wide = wide_rows(p.y_type, p.ldy);
  const int64_t n = n0 + wn * 16 * NT + 4 * NT * g;
  float sw[4 * NT];
  if (OP::SCALED) {
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) sw[i] = p.ws[(int64_t)t.e * p.N + min(n + i, p.N - 1)];
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = wm * 16 * MT + 16 * m + r;
    if (row >= t.n || n >= p.N) continue;
    float v[4 * NT];
    float sx = 1.0f;
    if (OP::SCALED) {
      const int at = row_of(p.perm, p.k_inv, p.T, p.k, t.p0 + row);
      sx = at < 0 ? 0.0f : p.xs[at];
    }
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) v[i] = OP::SCALED ? (float)acc[i / 4][m][i % 4] * sx * sw[i] : (float)acc[i / 4][m][i % 4];
    store_values<4 * NT>(p.y, p.y_type, (int64_t)(t.p0 + row) * p.ldy + n, p.N - n, wide, v);
  }
}

template <class OP, int BM, int BN, int WM, int WN, int NB>
hipError_t tiled(const Grouped &p, hipStream_t s) {
  const int64_t mt = grouped_max_tiles<BM>(p.offsets, p.E, p.P), nt = (p.N + BN - 1) / BN;
  hipLaunchKernelGGL((k_grouped<OP, BM, BN, WM, WN, NB>), dim3((unsigned)((mt * nt + 7) / 8 * 8)), dim3(64 * WM * WN), 0, s, p, (int)nt);
  return hipGetLastError();
}

template <class OP>
hipError_t choose(const Grouped &p, hipStream_t s) {
  return tiled<OP, 128, 128, 2, 2, 2>(p, s);
}

}  // namespace

hipError_t launch_grouped(const Grouped &p, hipStream_t s) {
  const int64_t mean = p.offsets ? p.P / p.E : p.P;  // rows of an expert
  if (mean <= 16) return launch_grouped_few(p, (int)(mean <= 8 ? 16 : 32), s);
  if (mean <= 64 && !p.offsets) return launch_grouped_few(p, (int)mean, s);
  if (p.type == DS4MOE_BF16) return choose<OpBf16>(p, s);
  if (p.type == DS4MOE_F16) return choose<OpF16>(p, s);
  return choose<OpI8>(p, s);
}

}  // namespace ds4
