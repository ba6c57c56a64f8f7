// Products of a few rows, grouped by expert or dense: the weights' bytes are
// what counts.
//
// Bound by reading the weights: 8 experts' 2048 x 4096 bf16 for one token, 134
// MB, 28.5 us (4.7 TB/s, the rate of a large copy); small ones by the launch.
//
// A workgroup has 16 weight rows and up to 16 MT rows of one expert; its eight
// waves share the columns and add up through LDS in a fixed order.  Weights
// and rows go from memory to the registers, where lane (r, g) holds bytes
// 32 g .. + 31 of 128 of row r (whole lines of memory): two matrix
// instructions, whose columns are then taken in another order, the same for
// both operands.
#include "grouped_dev.h"

namespace ds4 {

namespace {

constexpr int SW = 8;  // waves of a workgroup

template <class OP, int MT>
__global__ __launch_bounds__(64 * SW, 4) void k_grouped_few(Grouped p) {
  constexpr int U = MT == 1 ? 4 : 2;  // lines of a row on the way at a time
  __shared__ typename OP::Acc part[(SW - 1) * 64 * MT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  Finder f;
  f.load(p.offsets, p.E, p.P);
  f.set_height(16 * MT);
  if ((int)blockIdx.y >= f.count()) return;
  const Segment t = f.find(blockIdx.y);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  if (t.e < 0) {
    zero_rows(p.y, p.y_type, p.ldy, t.p0, t.n, n0, min(n0 + 16, p.N));
    return;
  }
  const char *const w = p.w + ((int64_t)t.e * p.N + min(n0 + r, p.N - 1)) * p.Kb;
  const char *x[MT];
  bool in[MT];
  int at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    at[m] = 16 * m + r < t.n ? row_of(p.perm, p.k_inv, p.T, t.p0 + 16 * m + r) : -1;
    in[m] = at[m] >= 0;
    x[m] = p.x + (in[m] ? at[m] : 0) * p.ldx;
  }
  typename OP::Acc acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = typename OP::Acc{0, 0, 0, 0};
  const int lines = (int)((p.Kb + 127) / 128);
  const u4 none = {0, 0, 0, 0};
  for (int c = U * wave; c < lines; c += SW * U) {
    u4 a[U][2], b[MT][U][2];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t o = (int64_t)(c + i) * 128 + 32 * g + 16 * h;
        const bool there = o < p.Kb;
        a[i][h] = there ? load16(w + o) : none;
#pragma unroll
        for (int m = 0; m < MT; ++m) b[m][i][h] = there && in[m] ? load16(x[m] + o) : none;
      }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = OP::mul(a[i][h], b[m][i][h], acc[m]);
  }
  if (wave) {
#pragma unroll
    for (int m = 0; m < MT; ++m) part[((wave - 1) * MT + m) * 64 + lane] = acc[m];
  }
  __syncthreads();
  if (wave) return;
  const int64_t n = n0 + 4 * g;
  const bool wide = p.ldy % 4 == 0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int i = 0; i < SW - 1; ++i) acc[m] += part[(i * MT + m) * 64 + lane];
    if (16 * m + r >= t.n || n >= p.N) continue;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = (float)acc[m][i];
      if (OP::SCALED) v[i] = v[i] * (in[m] ? p.xs[at[m]] : 0.0f) * p.ws[(int64_t)t.e * p.N + min(n + i, p.N - 1)];
    }
    store_values<4>(p.y, p.y_type, (int64_t)(t.p0 + 16 * m + r) * p.ldy + n, p.N - n, wide, v);
  }
}

template <class OP, int MT>
hipError_t few(const Grouped &p, hipStream_t s) {
  const dim3 g((unsigned)((p.N + 15) / 16), (unsigned)grouped_max_tiles(p.offsets != nullptr, p.E, p.P, 16 * MT));
  hipLaunchKernelGGL((k_grouped_few<OP, MT>), g, dim3(64 * SW), 0, s, p);
  return hipGetLastError();
}

}  // namespace

// Of an expert's rows a workgroup takes 16; of all rows of one matrix, up to
// 64, as many as there are, so that it is read once.
hipError_t launch_grouped_few(const Grouped &p, hipStream_t s) {
  if (p.type == DS4MOE_BF16) return few<OpBf16, 1>(p, s);
  if (p.type == DS4MOE_F16) return few<OpF16, 1>(p, s);
  if (p.offsets || p.P <= 16) return few<OpI8, 1>(p, s);
  return p.P <= 32 ? few<OpI8, 2>(p, s) : few<OpI8, 4>(p, s);
}

}  // namespace ds4
