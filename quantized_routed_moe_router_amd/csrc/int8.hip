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
unsigned groups(int64_t n, int64_t most = 1 << 20) { return (unsigned)(n < most ? n : most); }

// 8 adjacent values as they lie in memory: adjacent lanes read adjacent 16
// bytes of 16-bit values, and a row of 4096 of them takes a lane 32 registers
template <int TYPE>
struct Eight {
  static constexpr bool WIDE = TYPE == DS4MOE_F32;
  u4 u[WIDE ? 2 : 1];

  // from column c on, zeros past the end of `cols`; vec: aligned to 16 bytes
  __device__ __forceinline__ void load(const void *src, int64_t row, int64_t c, int64_t cols, bool vec) {
    if (vec && c + 8 <= cols) {
      u[0] = load16((const char *)src + (row + c) * (WIDE ? 4 : 2));
      if (WIDE) u[WIDE] = load16((const char *)src + (row + c) * 4 + 16);
      return;
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = c + i >= cols ? 0u : WIDE ? ((const uint32_t *)src)[row + c + i] : (uint32_t)((const uint16_t *)src)[row + c + i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (WIDE) {
        u[0][i] = w[i];
        u[WIDE][i] = w[4 + i];
      } else u[0][i] = w[2 * i] | w[2 * i + 1] << 16;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if (WIDE) return __uint_as_float(u[WIDE ? i >> 2 : 0][i & 3]);
    const uint32_t d = u[0][i >> 1];
    if (TYPE == DS4MOE_BF16) return __uint_as_float(i & 1 ? d & 0xFFFF0000u : d << 16);
    return half_bits_to_float((uint16_t)(i & 1 ? d >> 16 : d & 0xFFFFu));
  }
  // the largest magnitude so far as bits of the type, two halves side by side
  __device__ __forceinline__ uint32_t largest(uint32_t m) const {
    typedef uint16_t us2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (WIDE) {
        m = max(m, u[0][i] & 0x7FFFFFFFu);
        m = max(m, u[WIDE][i] & 0x7FFFFFFFu);
      } else
        m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, m), __builtin_bit_cast(us2, u[0][i] & 0x7FFF7FFFu)));
    }
    return m;
  }
  // and as bits of an fp32 number (NaN and infinity come out on top)
  static __device__ __forceinline__ uint32_t as_float(uint32_t m) {
    if (WIDE) return m;
    m = max(m & 0xFFFFu, m >> 16);
    return TYPE == DS4MOE_BF16 ? m << 16 : __float_as_uint(half_bits_to_float((uint16_t)m)) & 0x7FFFFFFFu;
  }
};

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

// codes of 8 values
template <int TYPE>
__device__ __forceinline__ u2 codes_of(const Eight<TYPE> &v, const RowScale &s) {
  constexpr float kShift = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer, which the low bits then are
  float off = s.up == 1.0f ? 0.0f : 1.0f;
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = v.value(i), u = fmaf(x, s.inv, kShift);
    q[i] = __float_as_uint(u);
    off = fmaxf(off, fabsf(fmaf(x, s.inv, kShift - u)));
  }
  if (off > 0.4999f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = (uint32_t)exact_code(v.value(i), s);
  }
  u2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0C0C0400) | __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x04000C0C);
  return o;
}

// L lanes to a row, 8 values a lane at a time; up to 8 steps stay in registers
// between the maximum and the codes, more are read again.  Up to 4096 columns a
// row is one wave's, which needs no barrier.  8192 x 4096 bf16 take 29.4 us (3.4
// TB/s of the bytes that go in and out; a copy reaches 4.9), 65536 x 4096 232 us
// (3.5).  Waves stand at waits for 79 % of their time, with 3 of them a SIMD on
// average; loading the next row under the codes of this one was not tried.
template <int TYPE, int L>
__global__ __launch_bounds__(256) void k_int8_quantize(int8_t *codes, float *scales, const void *src, int64_t rows, int64_t cols,
                                                       int64_t ld, bool vec) {
  constexpr int KEEP = L == 16 ? 2 : 8;
  __shared__ uint32_t tops[4];
  const int l = threadIdx.x % L;
  const int64_t to = (cols + 15) / 16 * 16;
  for (int64_t row0 = (int64_t)blockIdx.x * (256 / L); row0 < rows; row0 += (int64_t)gridDim.x * (256 / L)) {
    const int64_t row = row0 + threadIdx.x / L, at = row * ld;
    const bool in = row < rows;
    Eight<TYPE> v[KEEP];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int64_t c = (int64_t)(j * L + l) * 8;
      if (in && c < to) v[j].load(src, at, c, cols, vec);
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (in && (int64_t)(j * L + l) * 8 < to) m = v[j].largest(m);
    for (int64_t c = (int64_t)(KEEP * L + l) * 8; in && c < to; c += L * 8) {
      Eight<TYPE> u;
      u.load(src, at, c, cols, vec);
      m = u.largest(m);
    }
    m = Eight<TYPE>::as_float(m);
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
      const int64_t c = (int64_t)(j * L + l) * 8;
      if (c < to) *reinterpret_cast<u2 *>(codes + row * to + c) = codes_of(v[j], s);
    }
    for (int64_t c = (int64_t)(KEEP * L + l) * 8; c < to; c += L * 8) {
      Eight<TYPE> u;
      u.load(src, at, c, cols, vec);
      *reinterpret_cast<u2 *>(codes + row * to + c) = codes_of(u, s);
    }
    if (l == 0) scales[row] = s.scale;
  }
}

// 16 values a lane.  Bound by the memory: 8192 x 4096 to bf16 17.2 us (5.9 TB/s
// of codes and values, some of which stay in the cache), 65536 x 4096 138 us
// (5.8 TB/s).
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
  // Four workgroups a CU, which go round, against one for every row's place:
  // 8192 x 4096 29.4 us (32.2), 8192 x 1024 8.5 (9.9), 4096 x 16384 37.2
  // (41.2), 65536 x 4096 232 (237).  Short rows take sixteen: 100000 x 256 17.3
  // us (all 18.2, four 20.2).
  hipLaunchKernelGGL(f, dim3(groups((rows + per - 1) / per, cols <= 256 ? 4096 : 1024)), dim3(256), 0, s, codes, scales, src, rows, cols, ld, vec);
  return hipGetLastError();
}

// ---------------------------------------------------------------- products of a few rows, quantised on the way
// A workgroup of eight waves has 16 weight rows and all of the M <= 16 rows of
// a, which it quantises for itself: they come from L2, and a launch of their
// own takes longer.  The weights' first lines are asked for before that.  Then
// as the product of a few rows: the waves share the columns.  Bound by the
// launch and the latency of what follows another (a row, its maximum, the
// weights): one token, 2048 x 4096, 9.0 to 9.8 us a call, 1.7 of them for the
// weights' 8.4 MB.  In us, one launch and two: 2048 x 4096 1 row 9.0 and 11.9, 4
// 9.1 and 13.8, 8 11.8 and 14.2, 12 16.3 and 14.3; 8192 x 4096 1 row 10 and 17,
// 8 19 and 21, 12 26 and 22; 1001 x 2064 16 rows 10.7 and 11.6.  (16 rows of
// 4096 do not fit; beyond 8 rows of long matrices two launches are ahead.)
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
  constexpr int KEEP = 2;
  Eight<TYPE> v[KEEP];
  uint32_t m = 0;
  if (in) {
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if ((j * p.per + l) * 8 < K16) v[j].load(p.a, row * p.lda, (j * p.per + l) * 8, p.K, p.vec);
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if ((j * p.per + l) * 8 < K16) m = v[j].largest(m);
    for (int c = (KEEP * p.per + l) * 8; c < K16; c += p.per * 8) {
      Eight<TYPE> u;
      u.load(p.a, row * p.lda, c, p.K, p.vec);
      m = u.largest(m);
    }
  }
  m = Eight<TYPE>::as_float(m);
  for (int d = 1; d < min(p.per, 64); d *= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
    m = m > o ? m : o;
  }
  if (in && l % 64 == 0) atomicMax(&tops[row], m);
  __syncthreads();
  if (in) {
    const RowScale s = row_scale(tops[row]);
    if (l == 0) scales[row] = s.scale;
    char *const to = codes + row * step;
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if ((j * p.per + l) * 8 < K16) *reinterpret_cast<u2 *>(to + (j * p.per + l) * 8) = codes_of(v[j], s);
    for (int c = (KEEP * p.per + l) * 8; c < K16; c += p.per * 8) {
      Eight<TYPE> u;
      u.load(p.a, row * p.lda, c, p.K, p.vec);
      *reinterpret_cast<u2 *>(to + c) = codes_of(u, s);
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
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = (float)acc[i] * scales[r] * p.ws[min(n + i, p.N - 1)];
  store_values<4>(p.y, p.y_type, r * p.ldy + n, p.N - n, p.ldy % 4 == 0, y);
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
  // sixteen workgroups a CU, which go round, as long as there are few rounds
  // (8192 x 4096 17.2 us, one for every place 19.7; 100000 x 256 13.7, 16.2),
  // and one for every place beyond (65536 x 4096 138 us, going round 179)
  const int64_t all = (total + 255) / 256;
  hipLaunchKernelGGL(k_int8_dequantize, dim3(groups(all, all <= 16384 ? 4096 : 1 << 20)), dim3(256), 0, s, dst, type, ld, codes, scales, cols,
                     (uint32_t)per, total, wide);
  return hipGetLastError();
}

}  // namespace ds4
