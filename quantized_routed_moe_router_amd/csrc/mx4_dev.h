// Device-side pieces shared by the 4-bit microscaled kernels.
#pragma once
#include "common.h"
#include "mx4.h"

#include <type_traits>

namespace ds4 {

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef int i8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f4 mfma_bf16(bf8 a, bf8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// 16x16x128 product of two 4-bit operands; each lane gives the scale byte of
// its own block in bits 0-7 of sa and sb
__device__ __forceinline__ f4 mfma_mx4(u4 a, u4 b, f4 c, uint32_t sa, uint32_t sb) {
  const i8v A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i8v B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// The scale as the conversion takes it: a float of which only the exponent
// counts (exponent field 0 is 2^-127, 255 gives NaN).
__device__ __forceinline__ float scale_float(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 codes -> 8 bf16 times the scale: exact (two significant bits) as long as
// the value is a normal bf16 or a multiple of 2^-133
__device__ __forceinline__ bf8 codes_bf16(uint32_t c, float scale) {
  const bf2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ bf8 zero_bf8() {
  const u4 z = {0, 0, 0, 0};
  return __builtin_bit_cast(bf8, z);
}

__device__ __forceinline__ u4 load16(const void *p) { return *reinterpret_cast<const u4 *>(p); }

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// 4 adjacent values of the SwiGLU intermediate as PL bf16 terms, each the
// rounding of what the ones before it leave (planes `plane` elements apart)
template <int PL>
__device__ __forceinline__ void store_terms(uint16_t *p, int64_t plane, float v0, float v1, float v2, float v3) {
  float v[4] = {v0, v1, v2, v3};
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    bf4 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = (__bf16)v[i];
      v[i] = fabsf((float)b[i]) < INFINITY ? v[i] - (float)b[i] : 0.0f;
    }
    *reinterpret_cast<bf4 *>(p + q * plane) = b;
  }
}

// 16 bytes per lane from global memory into LDS without a register: lane l's
// bytes land at lds + 16 l (lds wave-uniform; inactive lanes write nothing)
__device__ __forceinline__ void load_lds16(const void *src, void *lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// dword g of the result: bytes g of the four dwords (block 4 s + g of a row of
// 16 scales goes to byte s of dword g)
__device__ __forceinline__ u4 transpose_bytes(u4 v) {
  const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05010400);  // a0 b0 a1 b1
  const uint32_t b = __builtin_amdgcn_perm(v[1], v[0], 0x07030602);
  const uint32_t c = __builtin_amdgcn_perm(v[3], v[2], 0x05010400);
  const uint32_t d = __builtin_amdgcn_perm(v[3], v[2], 0x07030602);
  return u4{__builtin_amdgcn_perm(c, a, 0x05040100), __builtin_amdgcn_perm(c, a, 0x07060302),
            __builtin_amdgcn_perm(d, b, 0x05040100), __builtin_amdgcn_perm(d, b, 0x07060302)};
}

// 16 scale bytes from block b on of a row of nblk; 127 past its end
__device__ __forceinline__ u4 scales16(const uint8_t *row, int b, int nblk) {
  u4 v;
  if (b + 16 <= nblk) {
    __builtin_memcpy(&v, row + b, 16);  // rows of scales lie at any byte
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i] |= (b + 4 * i + j < nblk ? (uint32_t)row[b + 4 * i + j] : 127u) << (8 * j);
    }
  }
  return v;
}

// four adjacent results of row m from column n on
template <bool YBF>
__device__ __forceinline__ void store_row4(const Mx4Product &p, int64_t m, int64_t n, f4 v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) {
      if (YBF) ((__bf16 *)p.y)[m * p.ldy + n + i] = (__bf16)v[i];
      else ((float *)p.y)[m * p.ldy + n + i] = v[i];
    }
}

// NV (4, 8 or 16) adjacent results of row m from column n on, n a multiple of
// NV; wide: rows are a multiple of 16 bytes apart
template <bool YBF, int NV>
__device__ __forceinline__ void store_cols(const Mx4Product &p, bool wide, int64_t m, int64_t n, const float (&v)[NV]) {
  if (wide && n + NV <= p.N) {
    if (YBF) {
      __bf16 *y = (__bf16 *)p.y + m * p.ldy + n;
#pragma unroll
      for (int i = 0; i < NV; i += 8) {
        if (NV == 4) *reinterpret_cast<bf4 *>(y) = bf4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        else
          *reinterpret_cast<bf8 *>(y + i) = bf8{(__bf16)v[i], (__bf16)v[i + 1], (__bf16)v[i + 2], (__bf16)v[i + 3],
                                                (__bf16)v[i + 4], (__bf16)v[i + 5], (__bf16)v[i + 6], (__bf16)v[i + 7]};
      }
    } else {
      float *y = (float *)p.y + m * p.ldy + n;
#pragma unroll
      for (int i = 0; i < NV; i += 4) *reinterpret_cast<f4 *>(y + i) = f4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (n + i < p.N) {
      if (YBF) ((__bf16 *)p.y)[m * p.ldy + n + i] = (__bf16)v[i];
      else ((float *)p.y)[m * p.ldy + n + i] = v[i];
    }
}
__device__ __forceinline__ bool wide_rows(const Mx4Product &p) { return p.ldy % (p.y_bf16 ? 8 : 4) == 0; }

// The workgroup's tile and weight rows.  Consecutive workgroups go to
// different XCDs, each of which takes a contiguous part of the work, all
// weight rows of a tile one after the other: a tile's activations stay in that
// XCD's L2, and neighbouring tiles (of one expert) share its weights there.
__device__ __forceinline__ bool tile_of(int id, int ntiles, int nrows, int &tile, int &nb) {
  const int all = ntiles * nrows, per = (all + 7) / 8, j = id >> 3, at = (id & 7) * per + j;
  tile = at / nrows;
  nb = at - tile * nrows;
  return j < per && at < all;
}
inline unsigned tile_grid(int64_t ntiles, int64_t nrows) { return (unsigned)((ntiles * nrows + 7) / 8 * 8); }

// Codes are loaded four lanes to a row (lane l: row l / 4, block l % 4), 64
// adjacent bytes that memory serves in one piece; a matrix instruction wants
// lane (r, g) = (l % 16, l / 16) to hold block g of row r.  The cross-lane
// read takes them there: with the lanes' own order every lane is a piece of
// its own.  For the gate/up product of 2048 tokens that halved the L1's
// lookups (205 to 94 million), but they were not what bounds it: with the
// codes of two stages asked for together the experts took 1108 us for 1117
// (with one term of the intermediate).
__device__ __forceinline__ u4 to_lanes(u4 v) {
  const int l = threadIdx.x & 63, from = ((l & 15) * 4 + (l >> 4)) * 4;
  u4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[i]);
  return o;
}

// Places of the 16-byte chunks of staged rows.  A 16-byte LDS read serves the
// lanes 0-3, 12-15, 20-23 and 24-27 together, then 4-7, 8-11, 16-19 and 28-31,
// and the same of the upper half; with these exchanges the rows that read
// chunk g and those that read g + 1 there lie in different banks (4.4 cycles a
// read; 8.1 with the row's own bits in their order, where they meet in pairs).
// r: row 0..15 of its group; chunk c goes to place c ^ f.
__device__ __forceinline__ int place8(int r) { return (r & 2) | (r >> 3) << 2; }                 // rows of 8 chunks
__device__ __forceinline__ int place16(int r) { return (r & 3) | ((4 - (r >> 2)) & 3) << 2; }  // rows of 16 chunks

// between LDS accesses of one wave, which execute in order: holds the compiler to it
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

// a workgroup barrier that leaves loads in flight (__syncthreads waits for
// all of them); LDS accesses before it are done
__device__ __forceinline__ void barrier_keep_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace ds4
