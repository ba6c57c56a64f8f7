// 8-bit integer values with one fp32 scale per row: quantisation and back.
//
// s = fp32(max|x| / 127), code = the nearest integer to x / s, ties to even,
// held to +-127.  The nearest integer to the exact quotient: q = rint(x (1/s))
// is at most one off next to a border, and the remainder x - q s, which a fused
// multiply-add gives without a rounding, says on which side.
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
__device__ __forceinline__ int code_of(float x, const RowScale &s) {
  x = s.up == 0.0f ? 0.0f : x * s.up;
  float q = rintf(x * s.inv);
  const float rest = fmaf(-q, s.unit, x), half = 0.5f * s.unit;
  const bool odd = (int)q & 1;
  if (rest > half || (rest == half && odd)) q += 1.0f;
  if (rest < -half || (rest == -half && odd)) q -= 1.0f;
  return min(max((int)q, -127), 127);
}

// L lanes to a row, 16 values a lane at a time; up to KEEP steps stay in
// registers between the maximum and the codes, more are read again.
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
    auto largest = [&](const float (&u)[16]) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t b = __float_as_uint(u[i]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
      }
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int64_t c = (int64_t)(j * L + l) * 16;
      if (in && c < cols) {
        load_values16<TYPE>(src, at, c, cols, vec, v[j]);
        largest(v[j]);
      }
    }
    for (int64_t c = (int64_t)(KEEP * L + l) * 16; in && c < cols; c += L * 16) {
      float u[16];
      load_values16<TYPE>(src, at, c, cols, vec, u);
      largest(u);
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
    auto put = [&](const float (&u)[16], int64_t c) {
      u4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) o[i] |= ((uint32_t)code_of(u[4 * i + b], s) & 255u) << (8 * b);
      }
      *reinterpret_cast<u4 *>(codes + row * to + c) = o;
    };
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int64_t c = (int64_t)(j * L + l) * 16;
      if (c < cols) put(v[j], c);
    }
    for (int64_t c = (int64_t)(KEEP * L + l) * 16; c < cols; c += L * 16) {
      float u[16];
      load_values16<TYPE>(src, at, c, cols, vec, u);
      put(u, c);
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
  auto f = cols <= 256 ? k_int8_quantize<TYPE, 16> : cols <= 2048 ? k_int8_quantize<TYPE, 64> : k_int8_quantize<TYPE, 256>;
  const int64_t per = cols <= 256 ? 16 : cols <= 2048 ? 4 : 1;
  hipLaunchKernelGGL(f, dim3(groups((rows + per - 1) / per)), dim3(256), 0, s, codes, scales, src, rows, cols, ld, vec);
  return hipGetLastError();
}

}  // namespace

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
