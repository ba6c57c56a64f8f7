// Products with both operands in 4-bit microscaled form, many rows: scaled
// matrix instructions of 16 x 16 x 128, which take the codes as they lie and
// one scale byte per lane's block.
//
// A workgroup of four waves has 16 MT activation rows and 64 NT weight rows.
// Both operands' codes are staged in LDS, 256 columns (whole lines of memory)
// at a time and NB buffers deep, by loads that bypass the registers; a wave
// multiplies all the activation rows with its own 16 NT weight rows.  (Weights straight to
// registers come in the wrong order: a lane's row is not its neighbour's, and
// 64 lookups a load or as many cross-lane reads cost more than the LDS does.)
// Row 4 g' + v of its i-th group of 16 is row 4 NT g' + 4 i + v of them: a
// lane's results are then 4 NT adjacent columns, whole pieces of memory (two
// bytes at a time, the stores took a third of the kernel).
// The scales of 512 columns (16 bytes a row) are turned into the order of the
// lanes on their way through LDS: lane (r, g) then reads one dword with the
// scales of its block of four successive instructions, each of which picks
// its byte.
//
// 2048 x 4096 x 4096 takes 28.7 us (2.4 Pflop/s), of which a launch with no
// columns takes about 5; each further 128 columns cost 0.7 us, where the
// matrix instructions of the whole card need 0.31.  Two buffers leave room for
// two workgroups on a CU, one of which multiplies while the other waits for
// its stage: 128 x 128 with two buffers 28.7 us, 128 x 256 with two 31.1 and
// with three 31.0, 64 x 128 with three 37.9; with the waves two by two, which
// reads a fifth less from LDS, 28.  What is left are the loads into LDS and the
// barriers between stages: the matrix units are busy a fifth of the time.
#include "mx4_dev.h"

namespace ds4 {

namespace {

template <int S>
__device__ __forceinline__ f4 mfma_sel(u4 a, u4 b, f4 c, uint32_t sa, uint32_t sb) {
  const i8v A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i8v B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, S, (int)sa, S, (int)sb);
}

template <int MT, int NT, int NB, bool YBF, bool EVEN>
__global__ __launch_bounds__(256, 2) void k_mx4_gemm4(Mx4Product p, int mtiles, int ntiles) {
  constexpr int BM = 16 * MT, ROWS = BM + 64 * NT;  // activation rows, then weight rows
  constexpr int STAGE = ROWS * 128;                  // bytes of 256 columns of their codes
  constexpr int DMA = STAGE / 4096, SPT = (ROWS + 255) / 256;
  __shared__ __attribute__((aligned(16))) char lds[NB * STAGE + 2 * ROWS * 16];
  char *const lsc = lds + NB * STAGE;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  int ti, nb;
  if (!tile_of(blockIdx.x, mtiles, ntiles, ti, nb)) return;
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)nb * 64 * NT;
  const int nblk = (int)(p.K / 32), last = (nblk + 7) / 8 - 1;
  const int64_t cb = p.K / 2;

  // a row of the tile: an activation row or a weight row (past the end the last one, never stored)
  auto row_of = [&](int row, const uint8_t *a, const uint8_t *w, int64_t bytes) {
    if (row < BM) return a + (m0 + row < p.M ? m0 + row : p.M - 1) * bytes;
    return w + (n0 + row - BM < p.N ? n0 + row - BM : p.N - 1) * bytes;
  };
  // load q of a stage: 8 rows of 8 chunks; a weight row's place goes by its row in the instruction
  const uint8_t *src[DMA];
  int ch[DMA];
#pragma unroll
  for (int q = 0; q < DMA; ++q) {
    const int row = (q * 4 + wave) * 8 + (lane >> 3), wrow = row - BM;
    ch[q] = (lane & 7) ^ place8(row < BM ? row & 15 : (wrow / (4 * NT) & 3) << 2 | (wrow & 3));
    src[q] = row_of(row, (const uint8_t *)p.a, p.w, cb) + ch[q] * 16;
  }
  const uint8_t *sx[SPT];
#pragma unroll
  for (int q = 0; q < SPT; ++q) sx[q] = row_of(min(q * 256 + tid, ROWS - 1), p.a_scales, p.ws, nblk);

  auto load = [&](int st, char *to) {
    if (EVEN || st * 8 + 8 <= nblk) {
#pragma unroll
      for (int q = 0; q < DMA; ++q) load_lds16(src[q] + (int64_t)st * 128, to + (q * 4 + wave) * 1024);
    } else {
#pragma unroll
      for (int q = 0; q < DMA; ++q) {
        char *d = to + (q * 4 + wave) * 1024;
        if (st * 8 + ch[q] < nblk) load_lds16(src[q] + (int64_t)st * 128, d);
        else *reinterpret_cast<u4 *>(d + lane * 16) = u4{0, 0, 0, 0};
      }
    }
    asm volatile("" ::: "memory");
  };
  u4 sc[SPT];
  auto load_sc = [&](int st) {
#pragma unroll
    for (int q = 0; q < SPT; ++q) sc[q] = scales16(sx[q], st * 8, nblk);
  };
  auto put_sc = [&](int buf) {
#pragma unroll
    for (int q = 0; q < SPT; ++q)
      if (q * 256 + tid < ROWS) *reinterpret_cast<u4 *>(lsc + (buf * ROWS + q * 256 + tid) * 16) = transpose_bytes(sc[q]);
  };
  f4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f4{0, 0, 0, 0};
  uint32_t sa[MT], sw[NT];
  // this lane's row of the weights' first group; the chunk of a half goes to place (4 h + g) ^ f
  const int wr = wave * 16 * NT + 4 * NT * (r >> 2) + (r & 3);
  const int fa = r * 128, fw = (BM + wr) * 128, f0 = (g ^ place8(r)) * 16;
  load_sc(0);
  load(0, lds);
  if (NB > 2) load(min(1, last), lds + STAGE);
  put_sc(0);
  wait_vm<(NB - 2) * DMA>();
  barrier_keep_loads();
  int s = 0;
  const char *x = lds;
  char *in = lds + (NB - 1) * STAGE;
  // One stage.  Past the end the last one is loaded again, so that the waits
  // are for a fixed number of loads.
  auto stage = [&](auto S) {
    if (S == 0) {
      const char *const ls = lsc + (s & 2) / 2 * ROWS * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) sa[m] = *reinterpret_cast<const uint32_t *>(ls + (16 * m + r) * 16 + 4 * g);
#pragma unroll
      for (int i = 0; i < NT; ++i) sw[i] = *reinterpret_cast<const uint32_t *>(ls + (BM + wr + 4 * i) * 16 + 4 * g);
      load_sc(min(s + 2, last / 2 * 2));
    }
    load(min(s + NB - 1, last), in);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u4 w[NT], a[MT];
#pragma unroll
      for (int i = 0; i < NT; ++i) w[i] = *reinterpret_cast<const u4 *>(x + fw + i * 512 + (f0 ^ 64 * h));
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m] = *reinterpret_cast<const u4 *>(x + fa + m * 2048 + (f0 ^ 64 * h));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[i][m] = h ? mfma_sel<S + 1>(w[i], a[m], acc[i][m], sw[i], sa[m]) : mfma_sel<S>(w[i], a[m], acc[i][m], sw[i], sa[m]);
    }
    if (S == 2) put_sc((s & 2) / 2 ^ 1);
    wait_vm<(NB - 2) * DMA>();  // the next stage's codes have landed
    barrier_keep_loads();
    x = x + STAGE == lds + NB * STAGE ? lds : x + STAGE;
    in = in + STAGE == lds + NB * STAGE ? lds : in + STAGE;
    return ++s > last;
  };
  for (;;) {
    if (stage(std::integral_constant<int, 0>{})) break;
    if (stage(std::integral_constant<int, 2>{})) break;
  }
  wait_vm<0>();  // the last loads into LDS, before it is released
  const bool wide = wide_rows(p);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = m0 + 16 * m + r;
    if (row >= p.M) continue;
    float v[4 * NT];
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) v[i] = acc[i / 4][m][i % 4];
    store_cols<YBF, 4 * NT>(p, wide, row, n0 + wave * 16 * NT + 4 * NT * g, v);
  }
}

}  // namespace

template <int MT, int NT, int NB>
static hipError_t gemm4(const Mx4Product &p, hipStream_t s) {
  const int mt = (int)((p.M + 16 * MT - 1) / (16 * MT)), nt = (int)((p.N + 64 * NT - 1) / (64 * NT));
  const dim3 g(tile_grid(mt, nt)), b(256);
  auto f = p.y_bf16 ? (p.K % 256 ? k_mx4_gemm4<MT, NT, NB, true, false> : k_mx4_gemm4<MT, NT, NB, true, true>)
                    : (p.K % 256 ? k_mx4_gemm4<MT, NT, NB, false, false> : k_mx4_gemm4<MT, NT, NB, false, true>);
  hipLaunchKernelGGL(f, g, b, 0, s, p, mt, nt);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm4(const Mx4Product &p, hipStream_t s) {
  auto groups = [&](int mt, int nt) { return ((p.M + 16 * mt - 1) / (16 * mt)) * ((p.N + 64 * nt - 1) / (64 * nt)); };
  // N = K = 4096, in us, this tile against the next: 2048 rows (512 groups of 128 x 128) 27.7 and 37.9, 1024 rows
  // (256) 19.4 and 19.4, 512 rows (128) 17.2 and 14.4.
  if (groups(8, 2) > 256) return gemm4<8, 2, 2>(p, s);
  // 1024 rows (512 groups of 64 x 128) 19.4 and 25.1, 512 rows (256) 14.4 and 14.6, 256 rows (128) 11.1 and 9.8.
  if (groups(4, 2) >= 192) return gemm4<4, 2, 3>(p, s);
  return gemm4<4, 1, 3>(p, s);
}

}  // namespace ds4
