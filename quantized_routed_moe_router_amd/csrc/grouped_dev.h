// Device-side pieces of the products grouped by expert and of their gradients.
#pragma once
#include "../../include/ds4moe.h"
#include "grouped.h"
#include "grouped_plan.h"
#include "mx4_dev.h"

namespace ds4 {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));

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

// Loads into LDS by buffer descriptors: a lane's offset at or beyond the range
// reads zeros without touching memory, and the compiler counts LDS reads apart
// from these loads (behind loads into LDS by plain addresses it waits for all
// LDS reads at every one).
constexpr int64_t kRange = 0xFFFF0000;
constexpr uint32_t kNowhere = 0xFFFFFFF0u;
// the range of a descriptor over `bytes` bytes (none if there are less)
__device__ __forceinline__ uint32_t range_of(int64_t bytes) { return bytes < 0 ? 0u : bytes > kRange ? (uint32_t)kRange : (uint32_t)bytes; }
__device__ __forceinline__ void load_stage16(__amdgpu_buffer_rsrc_t r, void *lds, uint32_t off, int stage_off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, off, stage_off, 0, 0);
}

// the row of x of an entry of the permutation, or -1 where it names none;
// k_inv: ceil(2^31 / k), which gives entry / k exactly for entries below 2^27,
// and no less than it for others
__device__ __forceinline__ int row_named(uint32_t k_inv, int T, int entry) {
  const int t = (int)__umulhi(2u * (uint32_t)entry, k_inv);
  return ((entry >= 0) & (t < T)) ? t : -1;
}
// the row of x of position p
__device__ __forceinline__ int row_of(const int32_t *perm, uint32_t k_inv, int T, int p) {
  return perm ? row_named(k_inv, T, perm[p]) : p < T ? p : -1;
}

// rows p0 .. p0 + n - 1 of expert e (-1: of none)
struct Segment {
  int e, p0, n;
};

// An operand whose rows are the terms of the sum lies across: it is staged as
// it lies, 64 rows by the tile's columns, chunk c of 16 bytes of row j in the
// place c ^ across_place(j), and turned on the way to the registers by the
// LDS' transposing read, which gives lane i of 16 the column i of four rows.
// PAIRS: group m of a wave's groups of 16 columns has columns 32 (m / 2) + 8 a
// + 4 (m % 2) + b in the place 4 a + b, so that a lane's results of two groups
// are 8 adjacent columns; a read then uses half of every chunk that it touches,
// and takes twice as long.  Otherwise group m has columns 16 m ..
template <bool PAIRS>
__device__ __forceinline__ int across_place(int row) {
  return PAIRS ? (row & 3) << 2 : (row & 3) << 1 | (row & 8);
}
typedef __attribute__((address_space(3))) s4 lds_s4;
// (__restrict__: without it the compiler lets this read wait for all loads into LDS, where it orders nothing: the
// barrier behind the waits does)
__device__ __forceinline__ u2 read_turned(lds_s4 *__restrict__ at) {
  return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(at));
}
typedef __attribute__((address_space(3))) const char *lds_at;
// Where this lane reads group m of columns from chunk c0 on, of rows of `bytes` each.  The place of a chunk makes it
// another number for every group (of PAIRS, every pair), so it is worked out once and kept.
template <bool PAIRS>
__device__ __forceinline__ uint32_t across_at(int bytes, int c0, int m) {
  const int lane = threadIdx.x & 63, r = lane & 15, j = 8 * (lane >> 4) + (r >> 2);  // the first of four rows
  const int chunk = PAIRS ? c0 + 4 * (m >> 1) + (r & 3) : c0 + 2 * m + (r >> 1 & 1), half = PAIRS ? m & 1 : r & 1;
  return j * bytes + (chunk ^ across_place<PAIRS>(j)) * 16 + 8 * half;
}
// a fragment: rows j .. j + 3 and j + 4 .. j + 7
__device__ __forceinline__ u4 read_across(lds_at x, int bytes) {
  const u2 lo = read_turned((lds_s4 *)x), hi = read_turned((lds_s4 *)(x + 4 * bytes));
  return u4{lo[0], lo[1], hi[0], hi[1]};
}

// sum over this lane and the lanes before it, inside the vector unit
template <int CTRL, int ROWS>
__device__ __forceinline__ int lanes_before(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v += lanes_before<0x111, 0xF>(v);  // 1, 2, 4, 8 lanes before, in a row of 16
  v += lanes_before<0x112, 0xF>(v);
  v += lanes_before<0x114, 0xF>(v);
  v += lanes_before<0x118, 0xF>(v);
  v += lanes_before<0x142, 0xA>(v);  // the last lane of the row before, in rows 1 and 3
  return v + lanes_before<0x143, 0xC>(v);  // the last lane of the first half, in the second
}

// The tiles of up to `height` rows (a multiple of 16, up to 256) that the
// experts' segments make, and tile `mt` of them once it is known.  Every wave
// looks for itself: a lane has up to eight experts, whose loads go out
// together, and the lanes' sums are added up over the wave; that is cheaper
// than a kernel that writes a list down first.
// Offsets are held to 0..P, so that whatever they are no row outside the
// arrays is touched.  Rows before the first and behind the last expert's make
// tiles of their own (e = -1).
struct Finder {
  static constexpr int PER = GROUPED_EXPERTS / 64;
  int start[PER], rows[PER], lane_sum, incl, tiles, head, first, last;
  int E, P, per, height;
  uint32_t inv;  // ceil(2^32 / height): n / height for n < 2^24
  bool one;

  __device__ __forceinline__ int at(const int32_t *o, int e) const { return min(max(o[min(e, E)], 0), P); }

  __device__ __forceinline__ void load(const int32_t *offsets, int E_, int P_) {
    E = E_;
    P = P_;
    one = offsets == nullptr;
    if (one) return;
    const int lane = threadIdx.x & 63;
    per = (E + 63) / 64;
    int o[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i) o[i] = i <= per ? at(offsets, lane * per + i) : 0;
    first = at(offsets, 0);
    last = max(first, at(offsets, E));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      start[i] = o[i];
      rows[i] = i < per && lane * per + i < E ? max(o[i + 1] - o[i], 0) : 0;
    }
  }
  __device__ __forceinline__ void set_height(int h) {
    height = h;
    inv = (uint32_t)(((1ull << 32) + h - 1) / h);
  }
  __device__ __forceinline__ int up(int n) const { return n > 0 ? (int)__umulhi((uint32_t)(n - 1), inv) + 1 : 0; }
  __device__ __forceinline__ int lane_tiles() const {
    int n = up(rows[0]);
    if (per > 1) {  // more than 64 experts
#pragma unroll
      for (int i = 1; i < PER; ++i) n += up(rows[i]);
    }
    return n;
  }

  // the number of tiles
  __device__ __forceinline__ int count() {
    if (one) return tiles = up(P);
    lane_sum = lane_tiles();
    incl = wave_scan(lane_sum);
    tiles = __builtin_amdgcn_readlane(incl, 63);
    head = up(first);
    return tiles + head + up(P - last);
  }

  // The height that suits the numbers: tiles run in rounds of as many as the
  // card holds (2^LOG), and a round lasts about as long as for 80 rows more
  // than its tiles have (256 rows 97 us, 224 90, 192 82, 160 71, 128 59, of 64
  // stages).  The choice itself costs a workgroup a microsecond.
  template <int LOG, int N>
  __device__ __forceinline__ void choose_height(const int (&heights)[N], int ntiles) {
    int best = INT32_MAX, of = heights[0], n[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      set_height(heights[i]);
      n[i] = one ? up(P) : lane_tiles();
    }
    if (!one) {
#pragma unroll
      for (int i = 0; i < N; ++i) n[i] = __builtin_amdgcn_readlane(wave_scan(n[i]), 63);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // within 32 bits: 2^22 tiles or a few more, 2^8 times as many of offsets that do not ascend
      const int cost = ((n[i] * ntiles + (1 << LOG) - 1) >> LOG) * (heights[i] + 80);
      if (cost < best) {
        best = cost;
        of = heights[i];
      }
    }
    set_height(__builtin_amdgcn_readfirstlane(of));
  }

  __device__ __forceinline__ Segment find(int mt) const {
    if (one) return Segment{0, mt * height, min(height, P - mt * height)};
    if (mt >= tiles) {
      mt -= tiles;
      if (mt < head) return Segment{-1, mt * height, min(height, first - mt * height)};
      const int p0 = last + (mt - head) * height;
      return Segment{-1, p0, min(height, P - p0)};
    }
    const int lane = threadIdx.x & 63;
    const int from = __ffsll((unsigned long long)__ballot(incl > mt)) - 1;
    int at = mt - (incl - lane_sum), e = lane * per, p0 = start[0] + at * height, n = min(height, rows[0] - at * height);
    if (per > 1) {
      at -= up(rows[0]);
#pragma unroll
      for (int i = 1; i < PER; ++i) {
        const int t = up(rows[i]);
        if (at >= 0 && at < t) {
          e = lane * per + i;
          p0 = start[i] + at * height;
          n = min(height, rows[i] - at * height);
        }
        at -= t;
      }
    }
    return Segment{__builtin_amdgcn_readlane(e, from), __builtin_amdgcn_readlane(p0, from), __builtin_amdgcn_readlane(n, from)};
  }
};

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
  if constexpr (NV >= 4) if (wide && n >= NV) {
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
