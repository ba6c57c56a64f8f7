// 4-bit microscaled values (E2M1 codes in blocks of 32 with an E8M0 scale):
// quantisation, products, and the routed SwiGLU experts on such weights.
//
// Codes and scales lie row by row as a checkpoint holds them: code k of a row
// in nibble k % 2 of byte k / 2, one scale byte per 32 codes; byte X stands
// for 2^(X-127), 255 for NaN.  A lane that holds 16 bytes of codes holds one
// block, so every lane of a matrix instruction has one scale.
#include "mx4_dev.h"

namespace ds4 {

namespace {

// ---------------------------------------------------------------- quantise, dequantise
// n / d for n < 2^31 by a multiplication: m = ceil(2^(32+s) / d), 2^s >= d
struct FastDiv {
  uint32_t m, s, d;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{(uint32_t)((((1ull << s) - d) << 32) / d + 1), s, d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
  const uint32_t q = __umulhi(n, f.m);
  return (uint32_t)(((uint64_t)q + n) >> f.s);
}

// Four lanes per block of 32, 8 values each.  Scale exponent
// floor(log2 max) - 2 (the block's largest value lands in [4, 8), the grid
// ends at 6 and the conversion saturates), round to nearest even on the grid
// by the conversion instruction.  A block with a NaN or an infinity has scale
// NaN; a block of zeros the smallest scale.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void k_mx4_quantize(uint8_t *codes, uint8_t *scales, const void *src, int64_t cols,
                                                      int64_t ld, FastDiv quads, uint32_t total) {
  const uint32_t q = blockIdx.x * 256u + threadIdx.x;
  const bool in = q < total;
  const uint32_t row = in ? div_by(q, quads) : 0;
  const uint32_t col8 = in ? q - row * quads.d : 0;  // group of 8 columns
  const int64_t c0 = (int64_t)col8 * 8, at = (int64_t)row * ld + c0;
  float v[8];
  if (VEC && in && c0 + 8 <= cols) {
    if (BF16) {
      const u4 u = load16((const uint16_t *)src + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
      const f4 a = *reinterpret_cast<const f4 *>((const float *)src + at);
      const f4 b = *reinterpret_cast<const f4 *>((const float *)src + at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (in && c0 + i < cols)
        v[i] = BF16 ? bf16_bits_to_float(((const uint16_t *)src)[at + i]) : ((const float *)src)[at + i];
    }
  }
  // the largest magnitude as bits: NaN and infinity come out on top
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = m > b ? m : b;
  }
  uint32_t o = (uint32_t)__shfl_xor((int)m, 1);
  m = m > o ? m : o;
  o = (uint32_t)__shfl_xor((int)m, 2);
  m = m > o ? m : o;
  const bool bad = m >= 0x7F800000u;
  int e = (int)(m >> 23) - 2;  // biased exponent of the scale (subnormal maxima clamp)
  if (e < 0) e = 0;
  const float up = ldexpf(1.0f, 127 - e);  // 2^-X: the codes are the values times it
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = bad ? 0.0f : v[i] * up, b = bad ? 0.0f : v[i + 1] * up;
    switch (i) {
      case 0: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a, b, 1.0f, 0); break;
      case 2: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a, b, 1.0f, 1); break;
      case 4: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a, b, 1.0f, 2); break;
      default: c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a, b, 1.0f, 3); break;
    }
  }
  if (!in) return;
  *reinterpret_cast<uint32_t *>(codes + (int64_t)q * 4) = c;
  if ((col8 & 3) == 0) scales[q >> 2] = bad ? 255 : (uint8_t)e;
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void k_mx4_dequantize(void *dst, int64_t ld, const uint8_t *codes,
                                                        const uint8_t *scales, int64_t cols, FastDiv quads,
                                                        uint32_t total) {
  const uint32_t q = blockIdx.x * 256u + threadIdx.x;
  if (q >= total) return;
  const uint32_t row = div_by(q, quads), col8 = q - row * quads.d;
  const int64_t c0 = (int64_t)col8 * 8, at = (int64_t)row * ld + c0;
  const uint32_t c = *reinterpret_cast<const uint32_t *>(codes + (int64_t)q * 4);
  const uint32_t sb = scales[q >> 2];
  // the code's value times 2^X in two exact steps (2^-127 is subnormal)
  const float s1 = sb == 255 ? NAN : ldexpf(1.0f, (int)sb - 127);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t n = c >> (4 * i), mag = n & 7u;
    const float g = mag < 2 ? 0.5f * mag : ldexpf(1.0f + 0.5f * (mag & 1), (int)(mag >> 1) - 1);
    v[i] = (n & 8u ? -g : g) * s1;
  }
  if (VEC && c0 + 8 <= cols) {
    if (BF16) {
      bf8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = (__bf16)v[i];
      *reinterpret_cast<bf8 *>((__bf16 *)dst + at) = b;
    } else {
      *reinterpret_cast<f4 *>((float *)dst + at) = f4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f4 *>((float *)dst + at + 4) = f4{v[4], v[5], v[6], v[7]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + i < cols) {
      if (BF16) ((__bf16 *)dst)[at + i] = (__bf16)v[i];
      else ((float *)dst)[at + i] = v[i];
    }
}

// ---------------------------------------------------------------- products with few rows of activations
// A wave multiplies 16 weight rows with 16 activation rows over its share of
// k; the waves of a workgroup take turns along k (128 at a time) and add up
// through LDS.  Lane (r, g) = (l % 16, l / 16) holds block g of the 128
// codes of weight row r, and for the bf16 steps j = 0..3 the activations
// 32 g + 8 j .. + 7 of row r: the steps cover the 128 in another order, the
// same for both operands.
constexpr int SM_WAVES = 8;

struct WRow {
  const uint8_t *c, *s;  // codes and scales of this lane's weight row, null outside
};

// adds w[16 rows] x a[16 rows]^T over k-tiles kt = wave, wave + nw, ... of nk128; K a multiple of 32
template <bool MX4A>
__device__ __forceinline__ void small_dot(f4 &acc, const uint8_t *wc, const uint8_t *wsc, const uint8_t *ap,
                                          const uint8_t *asc, int64_t K, int wave, int nw) {
  const int g = (threadIdx.x >> 4) & 3;
  const int nt = (int)((K + 127) / 128);
  for (int kt = wave; kt < nt; kt += nw) {
    const int64_t blk = (int64_t)kt * 4 + g;
    const bool in = blk * 32 < K;
    u4 w = {0, 0, 0, 0};
    uint32_t sw = 127, sa = 127;
    if (in && wc) {
      w = load16(wc + blk * 16);
      sw = wsc[blk];
    }
    if (MX4A) {
      u4 a = {0, 0, 0, 0};
      if (in && ap) {
        a = load16(ap + blk * 16);
        sa = asc[blk];
      }
      acc = mfma_mx4(w, a, acc, sw, sa);
    } else {
      const float sf = scale_float(sw);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf8 x = zero_bf8();
        if (in && ap) x = __builtin_bit_cast(bf8, load16(ap + (blk * 32 + 8 * j) * 2));
        acc = mfma_bf16(codes_bf16(w[j], sf), x, acc);
      }
    }
  }
}

// adds the waves' partial tiles; the sum is left in wave 0's lanes
__device__ __forceinline__ void join_waves(f4 *part, f4 &acc, int wave, int nw) {
  const int lane = threadIdx.x & 63;
  __syncthreads();
  part[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave == 0)
    for (int i = 1; i < nw; ++i) acc += part[i * 64 + lane];
}

template <bool MX4A, bool YBF>
__global__ __launch_bounds__(64 * SM_WAVES) void k_mx4_small(Mx4Product p) {
  __shared__ f4 part[SM_WAVES * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, n = n0 + r;
  const uint8_t *wc = n < p.N ? p.w + n * (p.K / 2) : nullptr;
  const uint8_t *wsc = p.ws + n * (p.K / 32);
  for (int64_t m0 = (int64_t)blockIdx.y * 16; m0 < p.M; m0 += (int64_t)gridDim.y * 16) {
    const int64_t m = m0 + r;
    const uint8_t *ap = nullptr, *asc = nullptr;
    if (m < p.M) {
      ap = (const uint8_t *)p.a + (MX4A ? m * (p.K / 2) : m * p.lda * 2);
      if (MX4A) asc = p.a_scales + m * (p.K / 32);
    }
    f4 acc = {0, 0, 0, 0};
    small_dot<MX4A>(acc, wc, wsc, ap, asc, p.K, wave, SM_WAVES);
    join_waves(part, acc, wave, SM_WAVES);
    if (wave == 0 && m < p.M) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t nn = n0 + 4 * g + i;
        if (nn < p.N) {
          if (YBF) ((__bf16 *)p.y)[m * p.ldy + nn] = (__bf16)acc[i];
          else ((float *)p.y)[m * p.ldy + nn] = acc[i];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- routed experts, few tokens each
// The assignment that opens an expert's range of the permutation stands for
// the expert; the others have nothing to do.  All of the routing is held to
// its ranges before it addresses anything.
struct ExpertRange {
  int e, p0, n;
};
__device__ __forceinline__ ExpertRange expert_of(const Mx4Experts &p, int a) {
  const int A = p.T * p.k;
  ExpertRange r{p.idx[a], 0, 0};
  if (r.e < 0 || r.e >= p.E) return r;
  r.p0 = p.offsets[r.e];
  if (r.p0 < 0 || r.p0 >= A || p.perm[r.p0] != a) return r;
  const int n = p.counts[r.e];
  r.n = n < 0 ? 0 : n > A - r.p0 ? A - r.p0 : n;
  return r;
}

template <int PL>
__global__ __launch_bounds__(64 * SM_WAVES) void k_mx4_gateup_small(Mx4Experts p) {
  __shared__ f4 part[SM_WAVES * 64];
  const ExpertRange er = expert_of(p, blockIdx.x);
  if (er.n == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int A = p.T * p.k;
  const int n0 = blockIdx.y * 16;
  const int64_t row = (int64_t)er.e * p.I + n0 + r;
  const bool in = n0 + r < p.I;
  const uint8_t *gc = in ? p.gate + row * (p.H / 2) : nullptr, *uc = in ? p.up + row * (p.H / 2) : nullptr;
  const uint8_t *gs = p.gate_s + row * (p.H / 32), *us = p.up_s + row * (p.H / 32);
  for (int t0 = 0; t0 < er.n; t0 += 16) {
    const int pos = er.p0 + t0 + r;
    const uint8_t *xp = nullptr;
    if (t0 + r < er.n) {
      const int a = p.perm[pos];
      if (a >= 0 && a < A) xp = (const uint8_t *)(p.x + (int64_t)(a / p.k) * p.ldx);
    }
    f4 ag = {0, 0, 0, 0}, au = {0, 0, 0, 0};
    small_dot<false>(ag, gc, gs, xp, nullptr, p.H, wave, SM_WAVES);
    small_dot<false>(au, uc, us, xp, nullptr, p.H, wave, SM_WAVES);
    join_waves(part, ag, wave, SM_WAVES);
    join_waves(part, au, wave, SM_WAVES);
    if (wave == 0 && t0 + r < er.n && n0 + 4 * g < p.I) {
      store_terms<PL>(p.h + (int64_t)pos * p.I + n0 + 4 * g, (int64_t)A * p.I, silu_mul(ag[0], au[0]),
                      silu_mul(ag[1], au[1]), silu_mul(ag[2], au[2]), silu_mul(ag[3], au[3]));
    }
  }
}

template <int PL>
__global__ __launch_bounds__(64 * SM_WAVES) void k_mx4_down_small(Mx4Experts p) {
  __shared__ f4 part[SM_WAVES * 64];
  const ExpertRange er = expert_of(p, blockIdx.x);
  if (er.n == 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int A = p.T * p.k;
  const int n0 = blockIdx.y * 16;
  const int64_t row = (int64_t)er.e * p.H + n0 + r;
  const uint8_t *wc = n0 + r < p.H ? p.down + row * (p.I / 2) : nullptr;
  const uint8_t *wsc = p.down_s + row * (p.I / 32);
  for (int t0 = 0; t0 < er.n; t0 += 16) {
    const int pos = er.p0 + t0 + r;
    f4 acc = {0, 0, 0, 0};
    for (int q = 0; q < PL; ++q) {
      const uint8_t *hp = t0 + r < er.n ? (const uint8_t *)(p.h + ((int64_t)q * A + pos) * p.I) : nullptr;
      small_dot<false>(acc, wc, wsc, hp, nullptr, p.I, wave, SM_WAVES);
    }
    join_waves(part, acc, wave, SM_WAVES);
    if (wave == 0 && t0 + r < er.n && n0 + 4 * g < p.H) {
      const int a = p.perm[pos];
      if (a >= 0 && a < A) *reinterpret_cast<f4 *>(p.ya + (int64_t)a * p.H + n0 + 4 * g) = acc;
    }
  }
}

// y[t] = sum_j w[t,j] ya[t*k+j], in the order of the ranks
template <bool YBF>
__global__ __launch_bounds__(256) void k_mx4_combine(Mx4Experts p) {
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= p.H) return;
  f4 y = {0, 0, 0, 0};
  for (int j = 0; j < p.k; ++j) {
    const int64_t a = t * p.k + j;
    const int e = p.idx[a];
    if (e < 0 || e >= p.E) continue;
    y += *reinterpret_cast<const f4 *>(p.ya + a * p.H + c) * p.w[a];
  }
  if (YBF) {
    bf4 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = (__bf16)y[i];
    *reinterpret_cast<bf4 *>((__bf16 *)p.y + t * p.H + c) = b;
  } else {
    *reinterpret_cast<f4 *>((float *)p.y + t * p.H + c) = y;
  }
}

}  // namespace

// Rows in slabs of fewer than 2^31 groups of 8 columns.
template <typename F>
static hipError_t by_slabs(int64_t rows, int64_t quads, F launch) {
  const int64_t most = (((int64_t)1 << 31) - 1) / quads;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    launch(r, (uint32_t)(n * quads));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx4_quantize(uint8_t *codes, uint8_t *scales, const void *src, bool bf16, int64_t rows, int64_t cols,
                               int64_t ld, hipStream_t s) {
  const int64_t nb = (cols + 31) / 32, quads = nb * 4, size = bf16 ? 2 : 4;
  const bool vec = ld * size % 16 == 0 && (uintptr_t)src % 16 == 0;
  const FastDiv f = fast_div((uint32_t)quads);
  return by_slabs(rows, quads, [&](int64_t r, uint32_t total) {
    const dim3 g((total + 255) / 256), b(256);
    uint8_t *c = codes + r * nb * 16, *sc = scales + r * nb;
    const void *x = (const uint8_t *)src + r * ld * size;
    if (bf16 && vec) hipLaunchKernelGGL((k_mx4_quantize<true, true>), g, b, 0, s, c, sc, x, cols, ld, f, total);
    else if (bf16) hipLaunchKernelGGL((k_mx4_quantize<true, false>), g, b, 0, s, c, sc, x, cols, ld, f, total);
    else if (vec) hipLaunchKernelGGL((k_mx4_quantize<false, true>), g, b, 0, s, c, sc, x, cols, ld, f, total);
    else hipLaunchKernelGGL((k_mx4_quantize<false, false>), g, b, 0, s, c, sc, x, cols, ld, f, total);
  });
}

hipError_t launch_mx4_dequantize(void *dst, bool bf16, int64_t ld, const uint8_t *codes, const uint8_t *scales,
                                 int64_t rows, int64_t cols, hipStream_t s) {
  const int64_t nb = (cols + 31) / 32, quads = nb * 4, size = bf16 ? 2 : 4;
  const bool vec = ld * size % 16 == 0 && (uintptr_t)dst % 16 == 0;
  const FastDiv f = fast_div((uint32_t)quads);
  return by_slabs(rows, quads, [&](int64_t r, uint32_t total) {
    const dim3 g((total + 255) / 256), b(256);
    const uint8_t *c = codes + r * nb * 16, *sc = scales + r * nb;
    void *y = (uint8_t *)dst + r * ld * size;
    if (bf16 && vec) hipLaunchKernelGGL((k_mx4_dequantize<true, true>), g, b, 0, s, y, ld, c, sc, cols, f, total);
    else if (bf16) hipLaunchKernelGGL((k_mx4_dequantize<true, false>), g, b, 0, s, y, ld, c, sc, cols, f, total);
    else if (vec) hipLaunchKernelGGL((k_mx4_dequantize<false, true>), g, b, 0, s, y, ld, c, sc, cols, f, total);
    else hipLaunchKernelGGL((k_mx4_dequantize<false, false>), g, b, 0, s, y, ld, c, sc, cols, f, total);
  });
}

hipError_t launch_mx4_product(const Mx4Product &p, hipStream_t s) {
  if (!p.a_scales && p.M > 16) return launch_mx4_gemm(p, s);
  const int64_t mt = (p.M + 15) / 16;
  const dim3 g((unsigned)((p.N + 15) / 16), (unsigned)(mt < 65535 ? mt : 65535)), b(64 * SM_WAVES);
  if (p.a_scales && p.y_bf16) hipLaunchKernelGGL((k_mx4_small<true, true>), g, b, 0, s, p);
  else if (p.a_scales) hipLaunchKernelGGL((k_mx4_small<true, false>), g, b, 0, s, p);
  else if (p.y_bf16) hipLaunchKernelGGL((k_mx4_small<false, true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((k_mx4_small<false, false>), g, b, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_mx4_experts(const Mx4Experts &p, hipStream_t s) {
  const int A = p.T * p.k;
  const dim3 b(64 * SM_WAVES), gg(A, (p.I + 15) / 16), gd(A, (p.H + 15) / 16), gc(p.T, (p.H / 4 + 255) / 256);
  if (p.T > 16) {
    const hipError_t e = launch_mx4_gemm_experts(p, s);
    if (e != hipSuccess) return e;
  } else if (p.y_bf16) {
    hipLaunchKernelGGL((k_mx4_gateup_small<1>), gg, b, 0, s, p);
    hipLaunchKernelGGL((k_mx4_down_small<1>), gd, b, 0, s, p);
  } else {
    hipLaunchKernelGGL((k_mx4_gateup_small<3>), gg, b, 0, s, p);
    hipLaunchKernelGGL((k_mx4_down_small<3>), gd, b, 0, s, p);
  }
  if (p.y_bf16) hipLaunchKernelGGL((k_mx4_combine<true>), gc, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((k_mx4_combine<false>), gc, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace ds4
