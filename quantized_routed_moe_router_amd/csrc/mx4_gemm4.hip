// Products with both operands in 4-bit microscaled form, many rows: scaled
// matrix instructions of 16 x 16 x 128, which take the codes as they lie and
// one scale byte per lane's block.
//
// A workgroup of four waves has 16 MT activation rows and 64 NT weight rows.
// The activations' codes are staged in LDS, 256 columns at a time and two
// buffers deep, by loads that bypass the registers; each wave holds the codes
// of its own 16 NT weight rows in registers, one stage ahead.  The scales of
// 512 columns (16 bytes a row) are turned into the order of the lanes on their
// way through LDS: lane (r, g) then reads one dword with the scales of its
// block of four successive instructions, each of which picks its byte.
#include "mx4_dev.h"

namespace ds4 {

namespace {

template <int S>
__device__ __forceinline__ f4 mfma_sel(u4 a, u4 b, f4 c, uint32_t sa, uint32_t sb) {
  const i8v A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i8v B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, S, (int)sa, S, (int)sb);
}

template <int MT, int NT, bool YBF>
__global__ __launch_bounds__(256, MT *NT >= 32 ? 1 : 2) void k_mx4_gemm4(Mx4Product p, int mtiles, int ntiles) {
  constexpr int BM = 16 * MT, BN = 64 * NT;
  constexpr int HALF = BM * 64, STAGE = 2 * HALF;      // bytes of 128 and of 256 columns of the activations' codes
  constexpr int SROWS = BM + BN, SPT = (SROWS + 255) / 256;  // rows with scales, and per thread
  constexpr int DMA = (STAGE + 4095) / 4096;           // loads per wave and stage
  __shared__ __attribute__((aligned(16))) char lds[2 * STAGE + 2 * SROWS * 16];
  char *const lsc = lds + 2 * STAGE;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  int ti, nb;
  if (!tile_of(blockIdx.x, mtiles, ntiles, ti, nb)) return;
  const int64_t m0 = (int64_t)ti * BM, n0 = (int64_t)nb * BN;
  const int nblk = (int)(p.K / 32), nst = (nblk + 7) / 8, nss = (nst + 1) / 2;
  const int64_t cb = p.K / 2;

  // this lane's rows: activations to LDS (16 rows of 4 chunks per load; chunk c
  // of row r at place c ^ (r / 4 % 4), so that 8 lanes of a read meet 8 banks)
  const uint8_t *ax[DMA];
  int at_[DMA], half[DMA];
#pragma unroll
  for (int q = 0; q < DMA; ++q) {
    const int u = q * 4 + wave;                        // load of the stage: 1 KB
    half[q] = u * 1024 / HALF;
    const int row = (u * 1024 % HALF) / 64 + (lane >> 2);
    const int64_t m = m0 + row < p.M ? m0 + row : p.M - 1;
    at_[q] = (lane & 3) ^ ((row >> 2) & 3);
    ax[q] = (const uint8_t *)p.a + m * cb;
  }
  const uint8_t *wx[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t n = n0 + (int64_t)(wave * NT + i) * 16 + r;
    wx[i] = p.w + (n < p.N ? n : p.N - 1) * cb;
  }
  const uint8_t *sx[SPT];
#pragma unroll
  for (int q = 0; q < SPT; ++q) {
    const int row = q * 256 + tid;
    const int64_t m = m0 + row < p.M ? m0 + row : p.M - 1, n = n0 + row - BM < p.N ? n0 + row - BM : p.N - 1;
    sx[q] = row < BM ? p.a_scales + m * nblk : p.ws + n * nblk;
  }

  auto load_a = [&](int st, char *to) {
    if (st >= nst) st = nst - 1;  // past the end: as many loads, never used
#pragma unroll
    for (int q = 0; q < DMA; ++q) {
      const int u = q * 4 + wave;
      if (DMA * 4096 > STAGE && u * 1024 >= STAGE) continue;
      const int blk = (st * 2 + half[q]) * 4 + at_[q];
      if (st * 8 + 8 <= nblk || blk < nblk) load_lds16(ax[q] + (int64_t)blk * 16, to + u * 1024);
      else *reinterpret_cast<u4 *>(to + u * 1024 + lane * 16) = u4{0, 0, 0, 0};
    }
    asm volatile("" ::: "memory");  // the waits count the loads issued after these
  };
  auto load_w = [&](int st, u4 (&w)[NT][2]) {
    if (st >= nst) st = nst - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int blk = (st * 2 + h) * 4 + g, b = blk < nblk ? blk : nblk - 1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        w[i][h] = load16(wx[i] + (int64_t)b * 16);
        if (blk >= nblk) w[i][h] = u4{0, 0, 0, 0};
      }
    }
  };
  f4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f4{0, 0, 0, 0};
  uint32_t sa[MT], sw[NT];
  const int fo = 16 * (g ^ ((r >> 2) & 3));
  auto compute = [&](auto S, const char *x, const u4 (&w)[NT][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u4 a[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m] = *reinterpret_cast<const u4 *>(x + h * HALF + (16 * m + r) * 64 + fo);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[i][m] = h ? mfma_sel<S + 1>(w[i][h], a[m], acc[i][m], sw[i], sa[m]) : mfma_sel<S>(w[i][h], a[m], acc[i][m], sw[i], sa[m]);
    }
  };
  u4 w0[NT][2], w1[NT][2], sc[SPT];
  auto load_sc = [&](int ss) {
#pragma unroll
    for (int q = 0; q < SPT; ++q)
      if (q * 256 + tid < SROWS) sc[q] = scales16(sx[q], ss * 16, nblk);
  };
  auto put_sc = [&](int buf) {
#pragma unroll
    for (int q = 0; q < SPT; ++q)
      if (q * 256 + tid < SROWS) *reinterpret_cast<u4 *>(lsc + (buf * SROWS + q * 256 + tid) * 16) = transpose_bytes(sc[q]);
  };
  load_sc(0);
  load_a(0, lds);
  load_w(0, w0);
  put_sc(0);
  wait_vm<0>();
  barrier_keep_loads();
  for (int ss = 0; ss < nss; ++ss) {
    const char *const ls = lsc + (ss & 1) * SROWS * 16;
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] = *reinterpret_cast<const uint32_t *>(ls + (16 * m + r) * 16 + 4 * g);
#pragma unroll
    for (int i = 0; i < NT; ++i) sw[i] = *reinterpret_cast<const uint32_t *>(ls + (BM + (wave * NT + i) * 16 + r) * 16 + 4 * g);
    if (ss + 1 < nss) load_sc(ss + 1);
    load_a(2 * ss + 1, lds + STAGE);
    load_w(2 * ss + 1, w1);
    compute(std::integral_constant<int, 0>{}, lds, w0);
    wait_vm<2 * NT>();  // the next stage's activations have landed
    barrier_keep_loads();
    if (2 * ss + 1 == nst) break;
    load_a(2 * ss + 2, lds);
    load_w(2 * ss + 2, w0);
    compute(std::integral_constant<int, 2>{}, lds + STAGE, w1);
    if (ss + 1 < nss) put_sc((ss + 1) & 1);
    wait_vm<2 * NT>();
    barrier_keep_loads();
  }
  wait_vm<0>();  // loads into LDS, before it is released
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = m0 + 16 * m + r;
    if (row >= p.M) continue;
#pragma unroll
    for (int i = 0; i < NT; ++i) store_row4<YBF>(p, row, n0 + (wave * NT + i) * 16 + 4 * g, acc[i][m]);
  }
}

}  // namespace

template <int MT, int NT>
static hipError_t gemm4(const Mx4Product &p, hipStream_t s) {
  const int mt = (int)((p.M + 16 * MT - 1) / (16 * MT)), nt = (int)((p.N + 64 * NT - 1) / (64 * NT));
  const dim3 g(tile_grid(mt, nt)), b(256);
  if (p.y_bf16) hipLaunchKernelGGL((k_mx4_gemm4<MT, NT, true>), g, b, 0, s, p, mt, nt);
  else hipLaunchKernelGGL((k_mx4_gemm4<MT, NT, false>), g, b, 0, s, p, mt, nt);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm4(const Mx4Product &p, hipStream_t s) {
  auto groups = [&](int mt, int nt) { return ((p.M + 16 * mt - 1) / (16 * mt)) * ((p.N + 64 * nt - 1) / (64 * nt)); };
  if (groups(8, 4) >= 192) return gemm4<8, 4>(p, s);
  if (groups(4, 2) >= 192) return gemm4<4, 2>(p, s);
  return gemm4<2, 1>(p, s);
}

}  // namespace ds4
