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
// NaN; a block of zeros the smallest scale.  16 bytes of bf16 and 4 of codes
// per lane, adjacent for adjacent lanes: memory bounds it.  8192 x 4096 in
// bf16, 85 MB, takes 18.1 us (4.7 TB/s), and as long to dequantise.
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

// ---------------------------------------------------------------- routed experts: the sum
// y[t] = sum_j w[t,j] ya[t*k+j], in the order of the ranks: fp32 results of
// the experts, each read once.  2048 tokens, k = 8, H = 4096: 268 MB read and
// 17 written in 54 us (5.2 TB/s).  (Sums in place by atomics would save the
// pass and give results that change from call to call.)
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
  if (p.M <= (p.a_scales ? MX4_FEW_ROWS4 : MX4_FEW_ROWS)) return launch_mx4_product_few(p, s);
  return p.a_scales ? launch_mx4_gemm4(p, s) : launch_mx4_gemm(p, s);
}

hipError_t launch_mx4_experts(const Mx4Experts &p, hipStream_t s) {
  const hipError_t e = mx4_few(p.T, p.k, p.E) ? launch_mx4_experts_few(p, s) : launch_mx4_gemm_experts(p, s);
  if (e != hipSuccess || p.T <= MX4_ONE) return e;
  const dim3 g(p.T, (p.H / 4 + 255) / 256), b(256);
  if (p.y_bf16) hipLaunchKernelGGL((k_mx4_combine<true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((k_mx4_combine<false>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace ds4
