// Device-side pieces of the products grouped by expert and of their gradients.
#pragma once
#include "../../include/ds4moe.h"
#include "grouped.h"
#include "mx4_dev.h"

namespace ds4 {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

// Matrix instructions of 16 x 16 whose operands are 16 bytes a lane: row
// l % 16, bytes 16 (l / 16) .. of 64.  That is 32 columns of 16 bits or 64 of
// 8, in the same number of cycles, so one kernel takes all three types.
struct OpBf16 {
  typedef f4 Acc;
  static constexpr bool SCALED = false;
  static __device__ __forceinline__ f4 mul(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  }
};
struct OpF16 {
  typedef f4 Acc;
  static constexpr bool SCALED = false;
  static __device__ __forceinline__ f4 mul(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
};
struct OpI8 {
  typedef i4 Acc;
  static constexpr bool SCALED = true;
  static __device__ __forceinline__ i4 mul(u4 a, u4 b, i4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4, a), __builtin_bit_cast(i4, b), c, 0, 0, 0);
  }
};

// 16 bytes of zeros in memory, which rows and columns that are not there read
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// the row of x of position p, or -1 where the permutation names none
__device__ __forceinline__ int row_of(const int32_t *perm, uint32_t k_inv, int T, int k, int p) {
  if (!perm) return p < T ? p : -1;
  const int a = perm[p];
  const int t = k_inv ? (int)__umulhi((uint32_t)a, k_inv) : a;
  return a >= 0 && t < T ? t : -1;
}

// rows p0 .. p0 + n - 1 of expert e (-1: of none)
struct Segment {
  int e, p0, n;
};

// The tiles of up to BM rows that the experts' segments make, and tile `mt` of
// them once it is known.  Every wave looks for itself: a lane has up to eight
// experts, whose loads go out together, and the lanes' sums are added up over
// the wave; that is cheaper than a kernel that writes a list down first.
// Offsets are held to 0..P, so that whatever they are no row outside the
// arrays is touched.  Rows before the first and behind the last expert's make
// tiles of their own (e = -1).
template <int BM>
struct Finder {
  static constexpr int PER = GROUPED_EXPERTS / 64;
  int start[PER], rows[PER], lane_sum, incl, tiles, head, first, last;
  int E, P, per;
  bool one;

  __device__ __forceinline__ int at(const int32_t *o, int e) const { return min(max(o[min(e, E)], 0), P); }

  __device__ __forceinline__ int count(const int32_t *offsets, int E_, int P_) {
    E = E_;
    P = P_;
    one = offsets == nullptr;
    if (one) return tiles = (P + BM - 1) / BM;
    const int lane = threadIdx.x & 63;
    per = (E + 63) / 64;
    int o[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i) o[i] = i <= per ? at(offsets, lane * per + i) : 0;
    first = at(offsets, 0);
    last = at(offsets, E);
    lane_sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      start[i] = o[i];
      rows[i] = i < per && lane * per + i < E ? max(o[i + 1] - o[i], 0) : 0;
      lane_sum += (rows[i] + BM - 1) / BM;
    }
    incl = lane_sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    tiles = __builtin_amdgcn_readlane(incl, 63);
    head = (first + BM - 1) / BM;
    return tiles + head + (P - max(first, last) + BM - 1) / BM;
  }

  __device__ __forceinline__ Segment find(int mt) const {
    if (one) return Segment{0, mt * BM, min(BM, P - mt * BM)};
    if (mt >= tiles) {
      mt -= tiles;
      if (mt < head) return Segment{-1, mt * BM, min(BM, first - mt * BM)};
      const int p0 = max(first, last) + (mt - head) * BM;
      return Segment{-1, p0, min(BM, P - p0)};
    }
    const int lane = threadIdx.x & 63;
    const int from = __ffsll((unsigned long long)__ballot(incl > mt)) - 1;
    int at = mt - (incl - lane_sum), e = 0, p0 = 0, n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int t = (rows[i] + BM - 1) / BM;
      if (at >= 0 && at < t) {
        e = lane * per + i;
        p0 = start[i] + at * BM;
        n = min(BM, rows[i] - at * BM);
      }
      at -= t;
    }
    return Segment{__builtin_amdgcn_readlane(e, from), __builtin_amdgcn_readlane(p0, from), __builtin_amdgcn_readlane(n, from)};
  }
};
// what a grid has room for: the most tiles that E segments of P rows can make
template <int BM>
inline int64_t grouped_max_tiles(const int32_t *offsets, int64_t E, int64_t P) {
  return offsets ? P / BM + (P < E + 2 ? P : E + 2) : (P + BM - 1) / BM;
}

// The workgroup's row tile and column tile.  Consecutive workgroups go to
// different XCDs, each of which takes a contiguous part of the work; GM row
// tiles by all column tiles at a time, so that those that run together on an
// XCD share rows and columns in its L2.
template <int GM>
__device__ __forceinline__ bool place_tile(int id, int mtiles, int ntiles, int &mt, int &nt) {
  const int all = mtiles * ntiles, per = (all + 7) / 8, j = id >> 3, at = (id & 7) * per + j;
  const int group = at / (GM * ntiles), rem = at - group * GM * ntiles, gm = min(GM, mtiles - group * GM);
  if (j >= per || at >= all) return false;
  nt = rem / gm;
  mt = group * GM + rem - nt * gm;
  return true;
}

// NV adjacent results of a row from y on, the first n of them; wide: whole
// pieces of 16 bytes (or of NV values, if that is less)
template <int NV>
__device__ __forceinline__ void store_values(void *base, int type, int64_t at, int64_t n, bool wide, const float (&v)[NV]) {
  if (wide && n >= NV) {
    if (type == DS4MOE_F32) {
      float *y = (float *)base + at;
#pragma unroll
      for (int i = 0; i < NV; i += 4) *reinterpret_cast<f4 *>(y + i) = f4{v[i], v[i + 1], v[i + 2], v[i + 3]};
      return;
    }
    uint32_t u[NV / 2];
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      if (type == DS4MOE_BF16) u[i] = __builtin_bit_cast(uint32_t, bf2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
      else u[i] = __builtin_bit_cast(uint32_t, h2{(half_t)v[2 * i], (half_t)v[2 * i + 1]});
    }
    uint16_t *y = (uint16_t *)base + at;
    if (NV == 4) *reinterpret_cast<u2 *>(y) = u2{u[0], u[1]};
    else {
#pragma unroll
      for (int i = 0; i < NV / 2; i += 4) *reinterpret_cast<u4 *>(y + 2 * i) = u4{u[i], u[i + 1], u[i + 2], u[i + 3]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i < n) {
      if (type == DS4MOE_F32) ((float *)base)[at + i] = v[i];
      else if (type == DS4MOE_BF16) ((__bf16 *)base)[at + i] = (__bf16)v[i];
      else ((half_t *)base)[at + i] = (half_t)v[i];
    }
}
// whether rows `ld` values apart hold their pieces of 16 bytes aligned
__device__ __forceinline__ bool wide_rows(int type, int64_t ld) { return ld % (type == DS4MOE_F32 ? 4 : 8) == 0; }

// rows p0 .. p0 + n - 1, columns n0 .. n1 - 1 set to zero
__device__ __forceinline__ void zero_rows(void *y, int type, int64_t ld, int64_t p0, int n, int64_t n0, int64_t n1) {
  for (int i = 0; i < n; ++i)
    for (int64_t c = n0 + threadIdx.x; c < n1; c += blockDim.x) {
      if (type == DS4MOE_F32) ((float *)y)[(p0 + i) * ld + c] = 0.0f;
      else ((uint16_t *)y)[(p0 + i) * ld + c] = 0;
    }
}

}  // namespace ds4
