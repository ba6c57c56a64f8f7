// Products of a few rows of activations with 4-bit microscaled weights, and
// the routed experts of up to 16 tokens: the weights' bytes are what counts.
//
// A wave holds up to KT k-tiles (128 columns of 16 weight rows, 16 bytes or
// one block per lane) of NM groups of rows in registers, all of them asked
// for before the first is used, so that a CU has 64 KB and more on the way.
// The waves of a workgroup share k (or the experts of a token) and add up
// through LDS in a fixed order.  The matrix instructions have 16 columns for
// the tokens; four tokens at a time are staged in LDS and fill four of them.
//
// H = 4096, I = 2048, k = 8 of 256 experts, 13.4 MB each: 16 tokens (about 102
// experts, fp32 results) take 168 us for gate and up (5.3 TB/s) and 121 for
// down (3.7 TB/s; from 93 to 173 by the call, with LDS conflicts in 18% of the
// cycles); one token 18.8 us (3.8 TB/s) and 11.9, where the launch and the
// first loads' latency are 5 us of each.  H = 7168, two steps of the staged
// rows of gate and up and 98 KB of LDS, one workgroup a CU: 16 tokens 469 us
// (474 for their bytes at 5 TB/s), one token 55 (37).
#include "mx4_dev.h"

namespace ds4 {

namespace {

constexpr int SW = 8;          // waves of a workgroup
constexpr int MAXA = 256;      // assignments of a small batch
constexpr int FEW_TILES = 8;   // 128-column tiles and terms of a wave that its LDS holds (8 KB)

// This wave's LDS: the assignments of its expert.  The ballot of a match
// gives every lane its place.
struct Members {
  uint8_t a[MAXA];
};

// The expert of assignment a0 and the assignments that have it, ascending;
// n = 0 if a0 is not the first of them or its index is out of range.
__device__ __forceinline__ int find_members(const int32_t *__restrict__ idx, int A, int a0, int E, Members &mb, int &e) {
  const int lane = threadIdx.x & 63;
  int v[MAXA / 64];
#pragma unroll
  for (int i = 0; i < MAXA / 64; ++i) v[i] = 64 * i + lane < A ? idx[64 * i + lane] : -1;
  e = -1;
#pragma unroll
  for (int i = 0; i < MAXA / 64; ++i)
    if (a0 >> 6 == i) e = __builtin_amdgcn_readlane(v[i], a0 & 63);
  if (e < 0 || e >= E) return 0;
  int n = 0;
  bool first = true;
#pragma unroll
  for (int i = 0; i < MAXA / 64; ++i) {
    const uint64_t m = __ballot(v[i] == e);
    if (v[i] == e)
      mb.a[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] = (uint8_t)(64 * i + lane);
    if (n == 0 && m && 64 * i + __ffsll((unsigned long long)m) - 1 != a0) first = false;
    n += __popcll(m);
  }
  return first ? n : 0;
}

// NM groups of 16 weight rows with one lane offset; row r of the wave's lanes
// past the matrix's end reads the last row
template <int NM>
struct Rows {
  const uint8_t *w[NM], *s[NM];
  uint32_t wo[NM], so[NM];
};

template <int NM>
__device__ __forceinline__ void set_rows(Rows<NM> &R, int i, const uint8_t *w, const uint8_t *s, int64_t row0, int64_t N,
                                         int64_t K) {
  const int r = threadIdx.x & 15;
  if (row0 >= N) row0 = 0;
  R.w[i] = w + row0 * (K / 2);
  R.s[i] = s + row0 * (K / 32);
  const uint32_t l = (uint32_t)(row0 + r < N ? r : N - 1 - row0);
  R.wo[i] = l * (uint32_t)(K / 2);
  R.so[i] = l * (uint32_t)(K / 32);
}

// acc[i] += weight rows of group i times the n <= 16 activation rows over the
// k-tiles kt0, kt0 + step, ...  row(m): row m of the activations, whose PL
// terms lie `plane` bytes apart.  lds: PL * KT * 1024 bytes of this wave.
template <int NM, int KT, int PL, typename F>
__device__ __forceinline__ void small_dot(f4 (&acc)[NM], const Rows<NM> &R, int64_t K, int kt0, int step, int n, F row,
                                          int64_t plane, char *lds) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int nblk = (int)(K / 32), nt = (nblk + 3) / 4;
  for (int c = kt0; c < nt; c += step * KT) {
    u4 w[NM][KT];
    uint32_t sc[NM][KT];
    for (int m0 = 0; m0 < n; m0 += 4) {
      // piece l + 64 u of the stage: term, row, tile, 16-byte chunk
      __builtin_amdgcn_s_waitcnt(0xC07F);  // reads of the last stage are done
#pragma unroll
      for (int u = 0; u < PL * KT; ++u) {
        const int id = lane + 64 * u, ch = id & 15, i = (id >> 4) % KT, m = (id >> 4) / KT % 4, q = (id >> 6) / KT;
        const int64_t k = ((int64_t)c + (int64_t)step * i) * 128 + ch * 8;
        if (m0 + m < n) {
          char *to = lds + 1024 * u;
          if (k < K) load_lds16(row(m0 + m) + q * plane + k * 2, to);
          else *reinterpret_cast<u4 *>(to + 16 * lane) = u4{0, 0, 0, 0};
        }
      }
      asm volatile("" ::: "memory");  // the wait below counts the loads issued after these
      if (m0 == 0) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const int blk = (c + step * t) * 4 + g, b = blk < nblk ? blk : nblk - 1;
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            w[i][t] = load16(R.w[i] + (R.wo[i] + (uint32_t)b * 16u));
            sc[i][t] = R.s[i][R.so[i] + (uint32_t)b];
          }
        }
        wait_vm<2 * NM * KT>();
      } else {
        wait_vm<0>();
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);
      asm volatile("" ::: "memory");
      const bool mine = r >= m0 && r < m0 + 4 && r < n;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const bool out = (c + step * t) * 4 + g >= nblk;
        if (c + step * t >= nt) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf8 x[PL];
#pragma unroll
          for (int q = 0; q < PL; ++q) {
            x[q] = zero_bf8();
            if (mine) x[q] = *reinterpret_cast<const bf8 *>(lds + (((q * 4 + (r & 3)) * KT + t) * 16 + 4 * g + j) * 16);
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            const bf8 a = codes_bf16(out ? 0 : w[i][t][j], scale_float(out ? 127 : sc[i][t]));
#pragma unroll
            for (int q = 0; q < PL; ++q) acc[i] = mfma_bf16(a, x[q], acc[i]);
          }
        }
      }
    }
  }
}

// column r of a product plus columns r + D, ... r + (PL - 1) D
template <int D, int PL>
__device__ __forceinline__ f4 add_columns(f4 v) {
  f4 s = v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = __float_as_int(v[i]);
    if (PL > 1) s[i] += __int_as_float(__builtin_amdgcn_update_dpp(0, u, 0x100 + D, 0xF, 0xF, true));
    if (PL > 2) s[i] += __int_as_float(__builtin_amdgcn_update_dpp(0, u, 0x100 + 2 * D, 0xF, 0xF, true));
  }
  return s;
}

// acc += 16 weight rows times one activation row over all of k.  lds: PL * KT * 256 bytes of this wave.
// WIDE: K a multiple of 512, the scales of 4 tiles are loaded at once.
template <int KT, int PL, bool WIDE>
__device__ __forceinline__ void one_dot(f4 &acc, const Rows<1> &R, int64_t K, const uint8_t *x, int64_t plane, char *lds) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int nblk = (int)(K / 32), nt = (nblk + 3) / 4;
  const uint32_t lw = (uint32_t)(lane >> 2) * (uint32_t)(K / 2);  // rows come in whole groups of 16
  for (int c = 0; c < nt; c += KT) {
    __builtin_amdgcn_s_waitcnt(0xC07F);
#pragma unroll
    for (int u = 0; u < PL * KT / 4; ++u) {
      const int id = lane + 64 * u, ch = id & 15, i = (id >> 4) % KT, q = (id >> 4) / KT;
      const int64_t k = (int64_t)(c + i) * 128 + ch * 8;
      char *to = lds + 1024 * u;
      if (k < K) load_lds16(x + q * plane + k * 2, to);
      else *reinterpret_cast<u4 *>(to + 16 * lane) = u4{0, 0, 0, 0};
    }
    asm volatile("" ::: "memory");  // the wait below counts the loads issued after these
    u4 w[KT];
    uint32_t sc[KT / 4][4];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int blk = (c + t) * 4 + (lane & 3), sb = (c + t) * 4 + g;
      w[t] = load16(R.w[0] + (lw + (uint32_t)(blk < nblk ? blk : nblk - 1) * 16u));
      if (!WIDE) sc[t / 4][t % 4] = R.s[0][R.so[0] + (uint32_t)(sb < nblk ? sb : nblk - 1)];
    }
    if (WIDE)
#pragma unroll
      for (int t = 0; t < KT; t += 4) {
        const int b = (c + t) * 4;
        __builtin_memcpy(sc[t / 4], R.s[0] + (R.so[0] + (uint32_t)(b < nblk ? b : 0)), 16);
      }
    wait_vm<KT + (WIDE ? KT / 4 : KT)>();
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      if (c + t >= nt) continue;
      const bool out = !WIDE && (c + t) * 4 + g >= nblk;
      const uint32_t sb = sc[t / 4][t % 4];
      const float sf = WIDE ? scale_float((sb >> (8 * g)) & 255u) : scale_float(out ? 127 : sb);
      const u4 wl = to_lanes(w[t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf8 a = codes_bf16(out ? 0 : wl[j], sf);
        bf8 x8 = zero_bf8();  // column q: term q
        if (r < PL) x8 = *reinterpret_cast<const bf8 *>(lds + ((r * KT + t) * 16 + 4 * g + j) * 16);
        acc = mfma_bf16(a, x8, acc);
      }
    }
  }
  acc = add_columns<1, PL>(acc);
}

// the workgroup's sum of acc, wave by wave, in wave 0
template <int NM>
__device__ __forceinline__ void join_waves(f4 *part, f4 (&acc)[NM]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  if (wave)
#pragma unroll
    for (int i = 0; i < NM; ++i) part[((wave - 1) * NM + i) * 64 + lane] = acc[i];
  __syncthreads();
  if (wave == 0)
#pragma unroll
    for (int q = 0; q < SW - 1; ++q)
#pragma unroll
      for (int i = 0; i < NM; ++i) acc[i] += part[(q * NM + i) * 64 + lane];
}

// Streaming form for up to 4 activation rows: they are staged once, and the
// weights of nrt row tiles of NM groups go by, each step's loads on their way
// while the step before is multiplied.  A step is KT adjacent tiles of k,
// whole lines of memory.  With SPL = SW the waves share k, their steps
// alternate, and each stages its own part; with SPL = 1 every wave has row
// tiles of its own over all of k, and nothing to wait for.  Where a row's
// scales allow it (WIDE: their number a multiple of 4 KT) a lane loads those
// of a step at once and picks its block's.  The terms of the activations take
// columns of the matrix instruction that the few tokens leave free: column r
// is term r / 4 of token r % 4, and the terms' columns are added at the end
// (16 tokens with three terms: 316 us with an instruction per term, 284 so).
// xs: PL * 4 rows of nti * 256 bytes of LDS, this wave's or (SPL = 1) the
// workgroup's.
template <int KT, int SPL>
inline __host__ __device__ int few_tiles(int64_t K) {  // staged tiles, whole steps
  return (int)((K / 32 + 4 * SPL * KT - 1) / (4 * SPL * KT)) * KT;
}

template <int KT, int PL, int SPL, typename F>
__device__ __forceinline__ void stage_rows(int64_t K, int wave, int n, F row, int64_t plane, char *xs) {
  const int lane = threadIdx.x & 63, nti = few_tiles<KT, SPL>(K);
  for (int u = SPL == 1 ? wave : 0; u < PL * nti; u += SPL == 1 ? SW : 1) {
    const int id = lane + 64 * u, ch = id & 15, i = (id >> 4) % nti, m = (id >> 4) / nti % 4, q = (id >> 6) / nti;
    const int64_t k = (int64_t)(SPL == 1 ? i : KT * (wave + SW * (i / KT)) + i % KT) * 128 + ch * 8;
    char *to = xs + 1024 * u;
    if (m < n) {
      if (k < K) load_lds16(row(m) + q * plane + k * 2, to);
      else *reinterpret_cast<u4 *>(to + 16 * lane) = u4{0, 0, 0, 0};
    }
  }
  asm volatile("" ::: "memory");  // the waits count the loads issued after these
}

template <int NM, int KT, bool WIDE>
struct Ahead {
  u4 w[NM][KT];
  uint32_t s[NM][KT];  // WIDE: the scales of tile t, one byte per block; else this lane's
};

// scale bytes [b, b + 4 KT) of a row
template <int KT>
__device__ __forceinline__ void load_scales(const uint8_t *p, uint32_t (&s)[KT]) {
  static_assert(KT == 2 || KT % 4 == 0, "whole loads");
#pragma unroll
  for (int t = 0; t < KT; t += 4) __builtin_memcpy(s + t, p + 4 * t, KT == 2 ? 8 : 16);
}

template <int NM, int KT, int PL, int SPL, bool WIDE, typename B, typename D>
__device__ __forceinline__ void stream_rows(int64_t K, int wave, int nrt, int n, const char *xs, B base, D done) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int nblk = (int)(K / 32), nt = (nblk + 3) / 4, nti = few_tiles<KT, SPL>(K), nch = nti / KT, steps = nrt * nch;
  const uint32_t wo = (uint32_t)(lane >> 2) * (uint32_t)(K / 2), so = (uint32_t)r * (uint32_t)(K / 32);
  int rl = 0, cl = 0;  // row tile and step of the next loads
  auto load = [&](Ahead<NM, KT, WIDE> &a) {
    const int t0 = SPL == 1 ? KT * cl : KT * (wave + SW * cl);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const uint8_t *w, *s;
      base(i, rl, w, s);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const int blk = (t0 + t) * 4 + (lane & 3), b = blk < nblk ? blk : nblk - 1;
        a.w[i][t] = load16(w + (wo + (uint32_t)b * 16u));
        const int sb = (t0 + t) * 4 + g;
        if (!WIDE) a.s[i][t] = s[so + (uint32_t)(sb < nblk ? sb : nblk - 1)];
      }
      if (WIDE) load_scales<KT>(s + (so + (uint32_t)(t0 * 4 < nblk ? t0 * 4 : 0)), a.s[i]);
    }
    if (++cl == nch) {
      cl = 0;
      ++rl;
    }
  };
  f4 acc[NM];
  int rt = 0, c = 0;
  auto step = [&](const Ahead<NM, KT, WIDE> &a) {
    if (c == 0)
#pragma unroll
      for (int i = 0; i < NM; ++i) acc[i] = f4{0, 0, 0, 0};
    const int t0 = SPL == 1 ? KT * c : KT * (wave + SW * c);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      if (t0 + t >= nt) continue;
      const bool out = !WIDE && (t0 + t) * 4 + g >= nblk;
      float sf[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) sf[i] = WIDE ? scale_float((a.s[i][t] >> (8 * g)) & 255u) : scale_float(out ? 127 : a.s[i][t]);
      u4 wl[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) wl[i] = to_lanes(a.w[i][t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf8 x = zero_bf8();
        if (r < 4 * PL && (r & 3) < n) x = *reinterpret_cast<const bf8 *>(xs + (r * nti + c * KT + t) * 256 + (4 * g + j) * 16);
#pragma unroll
        for (int i = 0; i < NM; ++i) acc[i] = mfma_bf16(codes_bf16(out ? 0 : wl[i][j], sf[i]), x, acc[i]);
      }
    }
    if (++c == nch) {
      c = 0;
#pragma unroll
      for (int i = 0; i < NM; ++i) acc[i] = add_columns<4, PL>(acc[i]);
      done(rt++, acc);
    }
  };
  Ahead<NM, KT, WIDE> a0, a1;
  load(a0);
  wait_vm<NM * KT + (WIDE ? NM * ((KT + 3) / 4) : NM * KT)>();  // the activations are there
  if (SPL == 1) barrier_keep_loads();
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
  // no load in the loop hangs on a condition: a step then waits for its own
  // loads alone, and not for the next step's
  int q = 0;
  for (; q + 2 < steps; q += 2) {
    load(a1);
    step(a0);
    load(a0);
    step(a1);
  }
  if (q + 2 == steps) {
    load(a1);
    step(a0);
    step(a1);
  } else {
    step(a0);
  }
}

// the waves' sums of a row tile to one of them (each in its turn), which then
// has it in acc; part: two buffers of SW * NM * 64 values
template <int NM>
__device__ __forceinline__ bool join_tile(f4 *part, int rt, int wave, f4 (&acc)[NM]) {
  const int lane = threadIdx.x & 63;
  f4 *const b = part + (rt & 1) * SW * NM * 64;
#pragma unroll
  for (int i = 0; i < NM; ++i) b[(wave * NM + i) * 64 + lane] = acc[i];
  barrier_keep_loads();
  if (wave != (rt & (SW - 1))) return false;
#pragma unroll
  for (int i = 0; i < NM; ++i) acc[i] = b[i * 64 + lane];
#pragma unroll
  for (int q = 1; q < SW; ++q)
#pragma unroll
    for (int i = 0; i < NM; ++i) acc[i] += b[(q * NM + i) * 64 + lane];
  return true;
}

// ---------------------------------------------------------------- experts of up to 16 tokens
// h rows are the assignments here, so no permutation is needed: every wave
// finds its expert's tokens in the list of choices.
template <int PL>
__global__ __launch_bounds__(64 * SW) void k_mx4_gateup_few(Mx4Experts p, int nrt) {
  constexpr int KT = 4;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ f4 part[2 * SW * 2 * 64];
  __shared__ Members mb[SW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int A = p.T * p.k;
  int e;
  const int n = find_members(p.idx, A, blockIdx.y, p.E, mb[wave], e);
  if (n == 0) return;
  const int n0 = blockIdx.x * 16 * nrt, rts = min(nrt, (p.I - n0 + 15) / 16);
  const uint8_t *const ew[2] = {p.gate + (int64_t)e * p.I * (p.H / 2), p.up + (int64_t)e * p.I * (p.H / 2)};
  const uint8_t *const es[2] = {p.gate_s + (int64_t)e * p.I * (p.H / 32), p.up_s + (int64_t)e * p.I * (p.H / 32)};
  auto row = [&](int m) { return (const uint8_t *)(p.x + (int64_t)(mb[wave].a[m] / p.k) * p.ldx); };
  auto store = [&](int m, int rt, const f4 &u, const f4 &v) {
    store_terms<PL>(p.h + (int64_t)mb[wave].a[m] * p.I + n0 + 16 * rt + 4 * g, (int64_t)A * p.I, silu_mul(u[0], v[0]),
                    silu_mul(u[1], v[1]), silu_mul(u[2], v[2]), silu_mul(u[3], v[3]));
  };
  if (n <= 4 && few_tiles<KT, SW>(p.H) <= FEW_TILES) {
    char *const xs = lds + wave * few_tiles<KT, SW>(p.H) * 1024;
    stage_rows<KT, 1, SW>(p.H, wave, n, row, 0, xs);
    auto base = [&](int i, int rt, const uint8_t *&w, const uint8_t *&s) {
      w = ew[i] + (int64_t)(n0 + 16 * rt) * (p.H / 2);
      s = es[i] + (int64_t)(n0 + 16 * rt) * (p.H / 32);
    };
    auto done = [&](int rt, f4 (&acc)[2]) {
      if (join_tile<2>(part, rt, wave, acc) && r < n) store(r, rt, acc[0], acc[1]);
    };
    if (p.H % (128 * KT) == 0) stream_rows<2, KT, 1, SW, true>(p.H, wave, rts, n, xs, base, done);
    else stream_rows<2, KT, 1, SW, false>(p.H, wave, rts, n, xs, base, done);
    return;
  }
  for (int rt = 0; rt < rts; ++rt) {
    Rows<2> R;
#pragma unroll
    for (int i = 0; i < 2; ++i) set_rows(R, i, ew[i], es[i], n0 + 16 * rt, p.I, p.H);
    for (int m0 = 0; m0 < n; m0 += 16) {
      f4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
      small_dot<2, KT, 1>(acc, R, p.H, wave, SW, min(n - m0, 16), [&](int m) { return row(m0 + m); }, 0, lds + wave * KT * 1024);
      join_waves<2>(part, acc);
      if (wave == 0 && m0 + r < n) store(m0 + r, rt, acc[0], acc[1]);
    }
  }
}

template <int PL>
__global__ __launch_bounds__(64 * SW) void k_mx4_down_few(Mx4Experts p, int nrt) {
  constexpr int KT = 8;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ Members mb[SW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int A = p.T * p.k;
  int e;
  const int n = find_members(p.idx, A, blockIdx.y, p.E, mb[wave], e);
  if (n == 0) return;
  const uint8_t *const ew = p.down + (int64_t)e * p.H * (p.I / 2), *const es = p.down_s + (int64_t)e * p.H * (p.I / 32);
  auto row = [&](int m) { return (const uint8_t *)(p.h + (int64_t)mb[wave].a[m] * p.I); };
  auto store = [&](int m, int c, const f4 &acc) {
    if (c < p.H) *reinterpret_cast<f4 *>(p.ya + (int64_t)mb[wave].a[m] * p.H + c + 4 * g) = acc;
  };
  if (n <= 4 && PL * few_tiles<KT, 1>(p.I) <= SW * FEW_TILES) {
    const int n0 = (blockIdx.x * SW + wave) * 16 * nrt;  // the wave's rows
    stage_rows<KT, PL, 1>(p.I, wave, n, row, (int64_t)A * p.I * 2, lds);
    auto base = [&](int, int rt, const uint8_t *&w, const uint8_t *&s) {
      int c = n0 + 16 * rt;
      if (c >= p.H) c = 0;  // past the end: read, never stored
      w = ew + (int64_t)c * (p.I / 2);
      s = es + (int64_t)c * (p.I / 32);
    };
    auto done = [&](int rt, f4 (&acc)[1]) {
      if (r < n) store(r, n0 + 16 * rt, acc[0]);
    };
    if (p.I % (128 * KT) == 0) stream_rows<1, KT, PL, 1, true>(p.I, wave, nrt, n, lds, base, done);
    else stream_rows<1, KT, PL, 1, false>(p.I, wave, nrt, n, lds, base, done);
    return;
  }
  f4 *const part = reinterpret_cast<f4 *>(lds + SW * PL * 2 * 1024);
  for (int rt = 0; rt < SW * nrt; ++rt) {
    const int c = (blockIdx.x * SW * nrt + rt) * 16;
    if (c >= p.H) break;
    Rows<1> R;
    set_rows(R, 0, ew, es, c, p.H, p.I);
    for (int m0 = 0; m0 < n; m0 += 16) {
      f4 acc[1] = {{0, 0, 0, 0}};
      small_dot<1, 2, PL>(acc, R, p.I, wave, SW, min(n - m0, 16), [&](int m) { return row(m0 + m); }, (int64_t)A * p.I * 2,
                          lds + wave * PL * 2 * 1024);
      join_waves<1>(part, acc);
      if (wave == 0 && m0 + r < n) store(m0 + r, c, acc[0]);
    }
  }
}

// Down projection and weighted sum of one token: each wave takes experts of
// the token, whole rows of k, and the first wave adds them up in the order of
// the ranks.  One launch and no results of single experts in memory: 11.8 us
// for one token and 36 MB.
template <int PL, bool YBF>
__global__ __launch_bounds__(64 * SW) void k_mx4_down_one(Mx4Experts p) {
  constexpr int KT = 16;
  __shared__ __attribute__((aligned(16))) char lds[SW * PL * KT * 256];
  __shared__ f4 part[16][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int t = blockIdx.y, n0 = blockIdx.x * 16, A = p.T * p.k;
  for (int j = wave; j < p.k; j += SW) {
    const int a = t * p.k + j, e = p.idx[a];
    f4 acc[1] = {{0, 0, 0, 0}};
    if (e >= 0 && e < p.E) {
      Rows<1> R;
      set_rows(R, 0, p.down + (int64_t)e * p.H * (p.I / 2), p.down_s + (int64_t)e * p.H * (p.I / 32), n0, p.H, p.I);
      const uint8_t *h = (const uint8_t *)(p.h + (int64_t)a * p.I);
      char *const xs = lds + wave * PL * KT * 256;
      if (p.I % 512 == 0) one_dot<KT, PL, true>(acc[0], R, p.I, h, (int64_t)A * p.I * 2, xs);
      else one_dot<KT, PL, false>(acc[0], R, p.I, h, (int64_t)A * p.I * 2, xs);
      const float w = p.w[a];
      acc[0] *= w;
    }
    if (r == 0) part[j][g] = acc[0];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    f4 y = {0, 0, 0, 0};
    for (int j = 0; j < p.k; ++j) y += part[j][threadIdx.x];
    const int64_t at = (int64_t)t * p.H + n0 + 4 * threadIdx.x;
    if (YBF) *reinterpret_cast<bf4 *>((__bf16 *)p.y + at) = bf4{(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
    else *reinterpret_cast<f4 *>((float *)p.y + at) = y;
  }
}

// ---------------------------------------------------------------- product of up to 16 rows
// 16 activation rows from memory (L2 after the first workgroup) as the matrix
// instruction wants them, and 16 weight rows per workgroup; the waves share k.
// 1 x 4096 x 2048, 4.5 MB: 5.4 us, a launch and two waits for memory.
template <bool YBF>
__global__ __launch_bounds__(64 * SW) void k_mx4_product_few(Mx4Product p) {
  constexpr int KT = 4;
  __shared__ f4 part[(SW - 1) * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16;
  const int nblk = (int)(p.K / 32), nt = (nblk + 3) / 4;
  Rows<1> R;
  set_rows(R, 0, p.w, p.ws, n0, p.N, p.K);
  const bool in = m0 + r < p.M;
  const uint8_t *const a = (const uint8_t *)p.a + (m0 + r < p.M ? m0 + r : p.M - 1) * p.lda * 2;
  f4 acc[1] = {{0, 0, 0, 0}};
  for (int c = KT * wave; c < nt; c += SW * KT) {  // KT adjacent tiles
    u4 w[KT], x[KT][4];
    uint32_t sc[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int blk = (c + t) * 4 + g, b = blk < nblk ? blk : nblk - 1;
      w[t] = load16(R.w[0] + (R.wo[0] + (uint32_t)b * 16u));
      sc[t] = R.s[0][R.so[0] + (uint32_t)b];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[t][j] = load16(a + (int64_t)b * 64 + j * 16);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const bool out = (c + t) * 4 + g >= nblk;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf8 v = __builtin_bit_cast(bf8, x[t][j]);
        if (out || !in) v = zero_bf8();
        acc[0] = mfma_bf16(codes_bf16(out ? 0 : w[t][j], scale_float(out ? 127 : sc[t])), v, acc[0]);
      }
    }
  }
  join_waves<1>(part, acc);
  if (wave == 0 && in) store_row4<YBF>(p, m0 + r, n0 + 4 * g, acc[0]);
}

// both operands in 4 bits: one scaled matrix instruction per k-tile
template <bool YBF>
__global__ __launch_bounds__(64 * SW) void k_mx4_product_few4(Mx4Product p) {
  constexpr int KT = 4;
  __shared__ f4 part[(SW - 1) * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int nblk = (int)(p.K / 32), nt = (nblk + 3) / 4;
  Rows<2> R;
  set_rows(R, 0, p.w, p.ws, n0, p.N, p.K);
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  set_rows(R, 1, (const uint8_t *)p.a, p.a_scales, m0, p.M, p.K);
  f4 acc[1] = {{0, 0, 0, 0}};
  for (int c = wave; c < nt; c += SW * KT) {
    u4 w[2][KT];
    uint32_t sc[2][KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int blk = (c + SW * t) * 4 + g, b = blk < nblk ? blk : nblk - 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i][t] = load16(R.w[i] + (R.wo[i] + (uint32_t)b * 16u));
        sc[i][t] = R.s[i][R.so[i] + (uint32_t)b];
      }
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const bool out = (c + SW * t) * 4 + g >= nblk;
      if (c + SW * t >= nt) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (out) {
          w[i][t] = u4{0, 0, 0, 0};
          sc[i][t] = 127;
        }
      acc[0] = mfma_mx4(w[0][t], w[1][t], acc[0], sc[0][t], sc[1][t]);
    }
  }
  join_waves<1>(part, acc);
  if (wave == 0 && m0 + r < p.M) store_row4<YBF>(p, m0 + r, n0 + 4 * g, acc[0]);
}

}  // namespace

hipError_t launch_mx4_product_few(const Mx4Product &p, hipStream_t s) {
  const dim3 g((unsigned)((p.N + 15) / 16), (unsigned)((p.M + 15) / 16)), b(64 * SW);
  if (p.a_scales && p.y_bf16) hipLaunchKernelGGL(k_mx4_product_few4<true>, g, b, 0, s, p);
  else if (p.a_scales) hipLaunchKernelGGL(k_mx4_product_few4<false>, g, b, 0, s, p);
  else if (p.y_bf16) hipLaunchKernelGGL(k_mx4_product_few<true>, g, b, 0, s, p);
  else hipLaunchKernelGGL(k_mx4_product_few<false>, g, b, 0, s, p);
  return hipGetLastError();
}

// LDS: the staged rows of the streaming form, and no less than the other form's
static unsigned gateup_lds(int64_t K) {
  const int t = few_tiles<4, SW>(K);
  return (unsigned)(SW * 1024 * (t <= FEW_TILES && t > 4 ? t : 4));
}
static unsigned down_lds(int64_t K, int PL) {
  const int t = PL * few_tiles<8, 1>(K), least = SW * PL * 2 + SW;
  return (unsigned)(1024 * (t <= SW * FEW_TILES && t > least ? t : least));
}

hipError_t launch_mx4_experts_few(const Mx4Experts &p, hipStream_t s) {
  const int A = p.T * p.k;
  // row tiles one after the other: the more, the longer the stream, as long as every CU has two workgroups
  auto tiles = [&](int per) {
    int n = 4;
    while (n > 1 && (per + n - 1) / n * A < 512) n /= 2;
    return n;
  };
  const int tu = (p.I + 15) / 16, td = (p.H + 16 * SW - 1) / (16 * SW), nu = tiles(tu), nd = tiles(td);
  const dim3 b(64 * SW), gg((tu + nu - 1) / nu, A), gd((td + nd - 1) / nd, A), go((p.H + 15) / 16, p.T);
  if (p.y_bf16) hipLaunchKernelGGL(k_mx4_gateup_few<2>, gg, b, gateup_lds(p.H), s, p, nu);
  else hipLaunchKernelGGL(k_mx4_gateup_few<3>, gg, b, gateup_lds(p.H), s, p, nu);
  if (p.T <= MX4_ONE) {
    if (p.y_bf16) hipLaunchKernelGGL((k_mx4_down_one<2, true>), go, b, 0, s, p);
    else hipLaunchKernelGGL((k_mx4_down_one<3, false>), go, b, 0, s, p);
  } else {
    if (p.y_bf16) hipLaunchKernelGGL(k_mx4_down_few<2>, gd, b, down_lds(p.I, 2), s, p, nd);
    else hipLaunchKernelGGL(k_mx4_down_few<3>, gd, b, down_lds(p.I, 3), s, p, nd);
  }
  return hipGetLastError();
}

}  // namespace ds4
