// 8-bit integer values with one fp32 scale per row: quantisation and back, and
// the product of a few rows that are quantised on the way.
//
// s = fp32(max|x| / 127), code = the nearest integer to x / s, ties to even,
// held to +-127.  The nearest integer to the exact quotient: t = x (1/s) is off
// by less than 2^-16, so away from the halves rounding it gives the code, and
// next to them (one wave in five, per step) the remainder x - q s, which a
// fused multiply-add gives without a rounding, says on which side x lies.
#include "grouped_dev.h"

namespace ds4 {

namespace {

// workgroups of a launch; what is beyond goes round
unsigned groups(int64_t n) { return (unsigned)(n < (1 << 20) ? n : 1 << 20); }

template <int TYPE>
__device__ __forceinline__ float value_at(const void *src, int64_t i) {
  if (TYPE == DS4MOE_F32) return ((const float *)src)[i];
  if (TYPE == DS4MOE_BF16) return bf16_bits_to_float(((const uint16_t *)src)[i]);
  return (float)((const half_t *)src)[i];
}

// 16 adjacent values from column c on, zeros past the end of `cols`
template <int TYPE>
__device__ __forceinline__ void load_values16(const void *src, int64_t row, int64_t c, int64_t cols, bool vec, float (&v)[16]) {
  if (vec && c + 16 <= cols) {
    if (TYPE == DS4MOE_F32) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f4 u = *reinterpret_cast<const f4 *>((const float *)src + row + c + i);
#pragma unroll
        for (int l = 0; l < 4; ++l) v[i + l] = u[l];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        const u4 u = load16((const uint16_t *)src + row + c + i);
#pragma unroll
        for (int l = 0; l < 8; ++l) {
          const uint16_t b = (uint16_t)(u[l / 2] >> (16 * (l & 1)));
          v[i + l] = TYPE == DS4MOE_BF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = c + i < cols ? value_at<TYPE>(src, row + c + i) : 0.0f;
}

struct RowScale {
  float scale, unit, up, inv;  // codes are of up x in units of `unit` = up scale
};

// from the bits of the largest magnitude (NaN and infinity come out on top)
__device__ __forceinline__ RowScale row_scale(uint32_t m) {
  RowScale s;
  if (m >= 0x7F800000u) return RowScale{NAN, 1.0f, 0.0f, 0.0f};
  const float top = __uint_as_float(m);
  s.scale = fminf(top / 127.0f, 0x1.020406p121f);  // 127 of the largest scale stay below infinity
  if (m && s.scale == 0.0f) s.scale = __uint_as_float(1u);
  s.up = s.scale < 0x1p-64f ? 0x1p80f : 1.0f;  // out of the subnormals, exactly, for the reciprocal
  s.unit = s.scale * s.up;
  s.inv = m ? 1.0f / s.unit : 0.0f;
  return s;
}
// code of a value next to a border, or of a row whose scale is not an ordinary number
__device__ __forceinline__ int exact_code(float x, const RowScale &s) {
  x = s.up == 0.0f ? 0.0f : x * s.up;
  float q = rintf(x * s.inv);
  const float rest = fmaf(-q, s.unit, x), half = 0.5f * s.unit;
  const bool odd = (int)q & 1;
  if (rest > half || (rest == half && odd)) q += 1.0f;
  if (rest < -half || (rest == -half && odd)) q -= 1.0f;
  return min(max((int)q, -127), 127);
}

// the largest magnitude of some values, as bits
__device__ __forceinline__ uint32_t largest(uint32_t m, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = m > b ? m : b;
  }
  return m;
}

// codes of 16 values
__device__ __forceinline__ u4 codes_of(const float (&v)[16], const RowScale &s) {
  constexpr float kShift = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer, which the low bits then are
  float off = s.up == 1.0f ? 0.0f : 1.0f;
  uint32_t q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float u = fmaf(v[i], s.inv, kShift);
    q[i] = __float_as_uint(u);
    off = fmaxf(off, fabsf(fmaf(v[i], s.inv, kShift - u)));
  }
  if (off > 0.4999f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = (uint32_t)exact_code(v[i], s);
  }
  u4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0C0C0400), hi = __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x04000C0C);
    o[i] = lo | hi;
  }
  return o;
}

// L lanes to a row, 16 values a lane at a time; up to KEEP steps stay in
// registers between the maximum and the codes, more are read again.  Up to 4096
// columns a row is one wave's, which needs no barrier.
template <int TYPE, int L>
__global__ __launch_bounds__(256) void k_int8_quantize(int8_t *codes, float *scales, const void *src, int64_t rows, int64_t cols,
                                                       int64_t ld, bool vec) {
  constexpr int KEEP = 4;
  __shared__ uint32_t tops[4];
  const int l = threadIdx.x % L;
  const int64_t to = (cols + 15) / 16 * 16;
  for (int64_t row0 = (int64_t)blockIdx.x * (256 / L); row0 < rows; row0 += (int64_t)gridDim.x * (256 / L)) {
    const int64_t row = row0 + threadIdx.x / L, at = row * ld;
    const bool in = row < rows;
    float v[KEEP][16];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int64_t c = (int64_t)(j * L + l) * 16;
      if (in && c < cols) load_values16<TYPE>(src, at, c, cols, vec, v[j]);
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (in && (int64_t)(j * L + l) * 16 < cols) m = largest(m, v[j]);
    for (int64_t c = (int64_t)(KEEP * L + l) * 16; in && c < cols; c += L * 16) {
      float u[16];
      load_values16<TYPE>(src, at, c, cols, vec, u);
      m = largest(m, u);
    }
#pragma unroll
    for (int d = 1; d < (L < 64 ? L : 64); d *= 2) {
      const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
      m = m > o ? m : o;
    }
    if (L > 64) {
      __syncthreads();  // the row before has read its maxima
      if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) m = m > tops[i] ? m : tops[i];
    }
    if (!in) continue;
    const RowScale s = row_scale(m);
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int64_t c = (int64_t)(j * L + l) * 16;
      if (c < cols) *reinterpret_cast<u4 *>(codes + row * to + c) = codes_of(v[j], s);
    }
    for (int64_t c = (int64_t)(KEEP * L + l) * 16; c < cols; c += L * 16) {
      float u[16];
      load_values16<TYPE>(src, at, c, cols, vec, u);
      *reinterpret_cast<u4 *>(codes + row * to + c) = codes_of(u, s);
    }
    if (l == 0) scales[row] = s.scale;
  }
}

// 16 values a lane
__global__ __launch_bounds__(256) void k_int8_dequantize(void *dst, int type, int64_t ld, const int8_t *codes, const float *scales,
                                                         int64_t cols, uint32_t per, int64_t total, bool wide) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, c = (i - row * per) * 16;
    const u4 u = load16(codes + i * 16);
    const float s = scales[row];
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = (float)((int)(u[j / 4] << (24 - 8 * (j & 3))) >> 24) * s;
    store_values<16>(dst, type, row * ld + c, cols - c, wide, v);
  }
}

template <int TYPE>
hipError_t quantize(int8_t *codes, float *scales, const void *src, int64_t rows, int64_t cols, int64_t ld, hipStream_t s) {
  const int64_t el = TYPE == DS4MOE_F32 ? 4 : 2;
  const bool vec = ((uintptr_t)src % 16) == 0 && (ld * el) % 16 == 0;
  auto f = cols <= 256 ? k_int8_quantize<TYPE, 16> : cols <= 4096 ? k_int8_quantize<TYPE, 64> : k_int8_quantize<TYPE, 256>;
  const int64_t per = cols <= 256 ? 16 : cols <= 4096 ? 4 : 1;
  hipLaunchKernelGGL(f, dim3(groups((rows + per - 1) / per)), dim3(256), 0, s, codes, scales, src, rows, cols, ld, vec);
  return hipGetLastError();
}

// ---------------------------------------------------------------- products of a few rows, quantised on the way
// A workgroup of eight waves has 16 weight rows and all of the M <= 16 rows of
// a, which it quantises for itself: they come from L2, and a launch of their
// own takes longer.  The weights' first lines are asked for before that.  Then
// as the product of a few rows: the waves share the columns.
constexpr int QW = 8;                    // waves
constexpr int QUANT_LDS = 64 << 10;      // bytes of codes

struct QuantProduct {
  void *y;
  int64_t ldy;
  int32_t y_type;
  const void *a;
  int64_t lda;
  const int8_t *w;
  const float *ws;
  int32_t M, per;  // threads of a row: 512 / (M up to a power of two)
  int64_t N, K;
  bool vec;
};

template <int TYPE>
__global__ __launch_bounds__(64 * QW, 4) void k_int8_few(QuantProduct p) {
  constexpr int U = 4;  // lines of 128 columns on the way at a time
  extern __shared__ __attribute__((aligned(16))) char codes[];
  __shared__ uint32_t tops[16];
  __shared__ float scales[16];
  __shared__ i4 part[(QW - 1) * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, K16 = (p.K + 15) / 16 * 16;
  const int step = (int)K16 + 16;  // rows of codes lie in different banks
  const int lines = (int)((K16 + 127) / 128);
  const int8_t *const w = p.w + min(n0 + r, p.N - 1) * K16;
  const u4 none = {0, 0, 0, 0};
  u4 b[U][2];
  auto weights = [&](int c) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t o = (int64_t)(c + i) * 128 + 32 * g + 16 * h;
        b[i][h] = o < K16 ? load16(w + o) : none;
      }
  };
  weights(U * wave);
  if (tid < 16) tops[tid] = 0;
  __syncthreads();
  const int row = tid / p.per, l = tid % p.per;
  const bool in = row < p.M;
  uint32_t m = 0;
  float first[16];
  if (in) {
    for (int64_t c = (int64_t)l * 16; c < p.K; c += p.per * 16) {
      float v[16];
      load_values16<TYPE>(p.a, row * p.lda, c, p.K, p.vec, v);
      m = largest(m, v);
      if (c == (int64_t)l * 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) first[i] = v[i];
      }
    }
  }
  for (int d = 1; d < min(p.per, 64); d *= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
    m = m > o ? m : o;
  }
  if (in && l % 64 == 0) atomicMax(&tops[row], m);
  __syncthreads();
  if (in) {
    const RowScale s = row_scale(tops[row]);
    if (l == 0) scales[row] = s.scale;
    for (int64_t c = (int64_t)l * 16; c < p.K; c += p.per * 16) {
      float v[16];
      if (c != (int64_t)l * 16) load_values16<TYPE>(p.a, row * p.lda, c, p.K, p.vec, v);
      *reinterpret_cast<u4 *>(codes + row * step + c) = c == (int64_t)l * 16 ? codes_of(first, s) : codes_of(v, s);
    }
  }
  __syncthreads();
  i4 acc = {0, 0, 0, 0};
  const char *const x = codes + r * step;
  for (int c = U * wave; c < lines; c += QW * U) {
    if (c != U * wave) weights(c);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = (c + i) * 128 + 32 * g + 16 * h;
        acc = OpI8::mul(b[i][h], ((r < p.M) & (o < K16)) ? *reinterpret_cast<const u4 *>(x + o) : none, acc);
      }
  }
  if (wave) part[(wave - 1) * 64 + lane] = acc;
  __syncthreads();
  const int64_t n = n0 + 4 * g;
  if (wave || r >= p.M || n >= p.N) return;
#pragma unroll
  for (int i = 0; i < QW - 1; ++i) acc += part[i * 64 + lane];
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)acc[i] * scales[r] * p.ws[min(n + i, p.N - 1)];
  store_values<4>(p.y, p.y_type, r * p.ldy + n, p.N - n, p.ldy % 4 == 0, v);
}

}  // namespace

bool int8_few_fits(int64_t M, int64_t K) { return M <= 16 && M * ((K + 15) / 16 * 16 + 16) <= QUANT_LDS; }

hipError_t launch_int8_few(const Grouped &g, const void *a, int32_t a_type, int64_t lda, int64_t K, hipStream_t s) {
  QuantProduct p{g.y, g.ldy, g.y_type, a, lda, (const int8_t *)g.w, g.ws, g.P, 64 * QW, g.N, K, false};
  for (int n = 1; n < g.P; n *= 2) p.per /= 2;
  const int64_t el = a_type == DS4MOE_F32 ? 4 : 2;
  p.vec = ((uintptr_t)a % 16) == 0 && (lda * el) % 16 == 0;
  auto f = a_type == DS4MOE_F32 ? k_int8_few<DS4MOE_F32> : a_type == DS4MOE_BF16 ? k_int8_few<DS4MOE_BF16> : k_int8_few<DS4MOE_F16>;
  const unsigned lds = (unsigned)(g.P * ((K + 15) / 16 * 16 + 16));
  hipLaunchKernelGGL(f, dim3((unsigned)((p.N + 15) / 16)), dim3(64 * QW), lds, s, p);
  return hipGetLastError();
}

hipError_t launch_int8_quantize(int8_t *codes, float *scales, const void *src, int32_t type, int64_t rows, int64_t cols, int64_t ld,
                                hipStream_t s) {
  if (type == DS4MOE_F32) return quantize<DS4MOE_F32>(codes, scales, src, rows, cols, ld, s);
  if (type == DS4MOE_BF16) return quantize<DS4MOE_BF16>(codes, scales, src, rows, cols, ld, s);
  return quantize<DS4MOE_F16>(codes, scales, src, rows, cols, ld, s);
}

hipError_t launch_int8_dequantize(void *dst, int32_t type, int64_t ld, const int8_t *codes, const float *scales, int64_t rows,
                                  int64_t cols, hipStream_t s) {
  const int64_t per = (cols + 15) / 16, total = rows * per, el = type == DS4MOE_F32 ? 4 : 2;
  const bool wide = ((uintptr_t)dst % 16) == 0 && (ld * el) % 16 == 0;
  hipLaunchKernelGGL(k_int8_dequantize, dim3(groups((total + 255) / 256)), dim3(256), 0, s, dst, type, ld, codes, scales, cols,
                     (uint32_t)per, total, wide);
  return hipGetLastError();
}

}  // namespace ds4
