// Expert gate: scores, groups, top-k, weights and the stable permutation from
// router logits, and the gradient of the weights.
//
// Mathematics, one token: s_e = sigmoid(l_e), softmax(l)_e or
// sqrt(softplus(l_e)); experts are ranked by s_e + b_e (by l_e where there is
// no bias: the same order without a rounding), groups of consecutive experts
// by the sum of their one or two best keys; the weights of the k best experts
// of the best groups are scale * s_j, divided by their sum where asked.
//
// 8192 tokens of 256 experts are 9 MB, 2 us of memory; what counts are the
// instructions of a token (790, of which the k rounds of a maximum over the
// wave and the scores are the larger parts) and their latency: each round is a
// chain of reduction, lane reads, ballot and shift, and with four waves on a
// SIMD instructions issue in less than half of the cycles.  A wave has the
// whole token in registers, so that no step waits for another wave, and two
// tokens of 8192.  Measured with 8 of 256 in 8 groups: 1 token 6.9 us, 8192
// tokens 16 us and 7 for the places, where each of 256 workgroups reads the
// counts of all 256 chunks again; 2048 tokens by softmax 8.3 and 5.2.
#include "mx4.h"
#include "route_dev.h"

namespace ds4 {

enum { SC_SQRT_SOFTPLUS = 0, SC_SIGMOID = 1, SC_SOFTMAX = 2 };

namespace {

constexpr int GATE_WAVES = 16;       // waves of a gate workgroup, one token each at a time
constexpr int GATE_MAXE = 512;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
  if (BF16) return bf16_bits_to_float(((const uint16_t *)p)[i]);
  return ((const float *)p)[i];
}

// NaN -> -inf (a masked expert); +inf -> the largest finite value, so that no
// difference or quotient of scores is a NaN
__device__ __forceinline__ float clean_logit(float l) {
  if (!(l >= -3.40282347e38f)) return -INFINITY;
  return fminf(l, 3.40282347e38f);
}

// sigmoid or sqrt(softplus) of one finite logit (0 for a masked one)
__device__ __forceinline__ float own_score(float l, int score) {
  if (l == -INFINITY) return 0.0f;
  if (score == SC_SIGMOID) return 1.0f / (1.0f + expf(-l));
  return l < -17.0f ? expf(0.5f * l) : router_score(l);  // e^l alone is subnormal from -87 on, its root is not
}

// Scores of chosen logits up to one common factor, for their quotients by
// their sum: below 0 a score goes with e^l (the root form with its root) and
// would end among the subnormals, so the factor e^max (its root) of the
// largest is taken out of all where that is below 0.  What is subnormal then
// has a subnormal weight.
__device__ __forceinline__ float relative_score(float l, int score, float max) {
  const float m = fminf(max, 0.0f);
  if (score == SC_SIGMOID) return expf(fminf(l, 0.0f) - m) / (1.0f + expf(-fabsf(l)));
  return l < -17.0f ? expf(0.5f * (l - m)) : router_score(l) * expf(-0.5f * m);
}

// order-preserving key of a float: every number >= 2, masked (-inf) 1
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 1u;
  return logit_key(v);
}

// Reductions by lane moves inside the vector unit: 4 steps in rows of 16
// lanes, 2 across them, the result read from the last lane.  (With reads of
// other lanes through the LDS unit, one after the other, the gate of 8192
// tokens took 22.5 us instead of 18.3.)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_move(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xF, false);
}
template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, uint32_t none, F f) {  // lane 15 of each row
  v = f(v, lane_move<0x111, 0xF>(none, v));
  v = f(v, lane_move<0x112, 0xF>(none, v));
  v = f(v, lane_move<0x114, 0xF>(none, v));
  return f(v, lane_move<0x118, 0xF>(none, v));
}
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t none, F f) {  // in every lane
  v = row_reduce(v, none, f);
  v = f(v, lane_move<0x142, 0xA>(none, v));
  v = f(v, lane_move<0x143, 0xC>(none, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t max_f32(uint32_t a, uint32_t b) {
  return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t add_f32(uint32_t a, uint32_t b) {
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}
constexpr uint32_t MINUS_INF = 0xFF800000u;
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) { return wave_reduce(v, 0u, max_u32); }
__device__ __forceinline__ float wave_max_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), MINUS_INF, max_f32));
}
__device__ __forceinline__ float wave_sum_f(float v) { return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, add_f32)); }
// of the first 16 lanes
__device__ __forceinline__ float first_max_f(float v) {
  return __int_as_float(__builtin_amdgcn_readlane((int)row_reduce(__float_as_uint(v), MINUS_INF, max_f32), 15));
}
__device__ __forceinline__ float first_sum_f(float v) {
  return __int_as_float(__builtin_amdgcn_readlane((int)row_reduce(__float_as_uint(v), 0u, add_f32), 15));
}

// the two largest of the lane's and another lane's two
template <int CTRL>
__device__ __forceinline__ void merge_move(float &m1, float &m2) {
  const float o1 = __uint_as_float(lane_move<CTRL, 0xF>(__float_as_uint(m1), __float_as_uint(m1)));
  const float o2 = __uint_as_float(lane_move<CTRL, 0xF>(__float_as_uint(m2), __float_as_uint(m2)));
  m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
  m1 = fmaxf(m1, o1);
}
__device__ __forceinline__ void merge_xor(float &m1, float &m2, int o) {
  const float o1 = __shfl_xor(m1, o), o2 = __shfl_xor(m2, o);
  m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
  m1 = fmaxf(m1, o1);
}

// the NK logits of a lane; VEC: in one load
template <int NK, bool BF16, bool VEC>
__device__ __forceinline__ void load_logits(const GateArgs &a, int64_t t, float (&x)[NK]) {
  const int e0 = NK * (threadIdx.x & 63);
  const int64_t at = t * a.ld + e0;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < NK; ++i) x[i] = -INFINITY;
    if (e0 >= a.E) return;
    if (BF16) {
      uint16_t u[NK];
      __builtin_memcpy(u, __builtin_assume_aligned((const uint16_t *)a.logits + at, 2 * NK), 2 * NK);
#pragma unroll
      for (int i = 0; i < NK; ++i) x[i] = clean_logit(bf16_bits_to_float(u[i]));
    } else {
      float u[NK];
      __builtin_memcpy(u, __builtin_assume_aligned((const float *)a.logits + at, NK < 4 ? 4 * NK : 16), 4 * NK);
#pragma unroll
      for (int i = 0; i < NK; ++i) x[i] = clean_logit(u[i]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NK; ++i) x[i] = e0 + i < a.E ? clean_logit(load_logit<BF16>(a.logits, at + i)) : -INFINITY;
}

// One token by one wave; lane l holds experts NK*l .. NK*l+NK-1.  Lane j < k
// returns expert and weight of rank j.  xl, kl: wave-private LDS rows of NK*64
// floats.
// b: the bias of the lane's experts.  Selection goes by scores of an ulp or
// two, as the weights do: the hardware's exponential alone, off by the
// rounding of its argument, is 16 ulp off at a logit of -40.
template <int NK>
__device__ __forceinline__ void gate_token(const GateArgs &a, const float (&x)[NK], const float (&b)[NK], float *xl,
                                           float *kl, int &my_e, float &my_w) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NK; ++i) xl[NK * lane + i] = x[i];
  // softmax over all experts: maximum and sum
  float mx = 0.0f, zinv = 1.0f, p[NK];
  const bool soft = a.score == SC_SOFTMAX;
  if (soft) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < NK; ++i) m = fmaxf(m, x[i]);
    mx = wave_max_f(m);
    float z = 0.0f;
    if (mx == -INFINITY) mx = 0.0f;  // every expert masked
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      p[i] = expf(x[i] - mx);
      z += p[i];
    }
    z = wave_sum_f(z);
    zinv = z > 0.0f ? 1.0f / z : 0.0f;
  }
  // value of each expert that the groups are ranked by (-inf where masked);
  // the experts are, too, where there is a bias, and by the logit otherwise
  const bool need_scores = a.bias != nullptr || (a.G > 1 && a.group_rank > 1);
  float v[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    v[i] = x[i];
    if (need_scores) {
      float c = soft ? p[i] * zinv : own_score(x[i], a.score);
      c += a.bias ? b[i] : 0.0f;
      v[i] = x[i] == -INFINITY || c != c ? -INFINITY : c;
    }
  }
  uint64_t stays = ~0ull;
  int lanes_per = 64;
  if (a.G > 1) {
#pragma unroll
    for (int i = 0; i < NK; ++i) kl[NK * lane + i] = v[i];
    wave_lds_order();
    // lanes_per lanes (a power of two) per group: the two best of the group
    lanes_per = 64 >> (32 - __clz(a.G - 1));
    const int g = lane / lanes_per, j = lane % lanes_per;
    float m1 = -INFINITY, m2 = -INFINITY;
    if (g < a.G)
      for (int i = j; i < a.per; i += lanes_per) {
        const float u = kl[g * a.per + i];
        m2 = fmaxf(m2, fminf(m1, u));
        m1 = fmaxf(m1, u);
      }
    if (lanes_per > 1) merge_move<0xB1>(m1, m2);   // neighbours
    if (lanes_per > 2) merge_move<0x4E>(m1, m2);   // pairs of a quad
    if (lanes_per > 4) merge_move<0x141>(m1, m2);  // quads of 8 lanes, mirrored
    if (lanes_per > 8) merge_move<0x140>(m1, m2);  // halves of a row, mirrored
    if (lanes_per > 16) merge_xor(m1, m2, 16);
    if (lanes_per > 32) merge_xor(m1, m2, 32);
    // a second best that is masked adds nothing; a group with none live is last
    const float gs = (a.group_rank > 1 && m2 > -INFINITY) ? m1 + m2 : m1;
    // groups before this one: a larger score, or an equal one and a lower index
    const uint32_t gk = order_key(gs);
    int rank = 0;
    for (int h = 0; h < a.G; ++h) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, h * lanes_per);
      rank += o > (h < g ? gk - 1 : gk) ? 1 : 0;
    }
    stays = __ballot(g < a.G && j == 0 && rank < a.top_groups);
  }
  uint32_t key[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int e = NK * lane + i;
    key[i] = 0u;
    if (e < a.E) {
      const int g = a.G > 1 ? (int)(((uint32_t)e * a.per_inv) >> 20) : 0;
      if (a.G <= 1 || ((stays >> (g * lanes_per)) & 1)) key[i] = order_key(a.bias ? v[i] : x[i]);
    }
  }
  // The lane's keys in descending order (equal ones as they are), then k
  // rounds of the wave's largest head: ties to the lowest lane, that is to the
  // lowest expert; the lane that has it moves its keys up.
  uint32_t slot[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) slot[i] = i;
#pragma unroll
  for (int p = 0; p < NK - 1; ++p)
#pragma unroll
    for (int i = 0; i < NK - 1 - p; ++i) {
      const bool up = key[i + 1] > key[i];
      const uint32_t k0 = key[i], s0 = slot[i];
      key[i] = up ? key[i + 1] : k0;
      key[i + 1] = up ? k0 : key[i + 1];
      slot[i] = up ? slot[i + 1] : s0;
      slot[i + 1] = up ? s0 : slot[i + 1];
    }
  int mine = 0;  // lane r: rank r's expert
  uint32_t my_key = 0u;
  for (int r = 0; r < a.k; ++r) {
    const uint32_t m = wave_max_u32(key[0]);
    const uint64_t at = __ballot(key[0] == m);
    const int win = __builtin_ctzll(at);
    const int e = NK * win + __builtin_amdgcn_readlane((int)slot[0], win);
    mine = lane == r ? e : mine;
    my_key = lane == r ? m : my_key;
    if (lane == win) {
#pragma unroll
      for (int i = 0; i < NK - 1; ++i) {
        key[i] = key[i + 1];
        slot[i] = slot[i + 1];
      }
      key[NK - 1] = 0u;
    }
  }
  my_e = mine;
  wave_lds_order();
  float s = 0.0f;
  const float l = lane < a.k ? xl[my_e] : -INFINITY;
  const bool live = lane < a.k && my_key > 1u && l != -INFINITY;
  if (a.renorm) mx = first_max_f(live ? l : -INFINITY);  // sums of the chosen alone
  if (live) {
    if (soft) s = expf(l - mx) * (a.renorm ? 1.0f : zinv);
    else s = a.renorm ? relative_score(l, a.score, mx) : own_score(l, a.score);
  }
  if (a.renorm) {
    const float S = first_sum_f(s);
    s = S > 0.0f ? s / S : 0.0f;
  }
  my_w = a.scale * s;
  wave_lds_order();
}

// exclusive prefix over `n` <= 512 ints in LDS by the first wave; total returned in every lane of it
__device__ __forceinline__ int wave_scan_512(const int32_t *c, int32_t *off, int n) {
  const int lane = threadIdx.x & 63;
  int v[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 8 * lane + i < n ? c[8 * lane + i] : 0;
    sum += v[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o);
    if (lane >= o) inc += u;
  }
  int run = inc - sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (8 * lane + i < n) off[8 * lane + i] = run;
    run += v[i];
  }
  return __shfl(inc, 63);
}

// One workgroup per chunk of tokens, a wave per token; a chunk's tokens go in
// blocks of 64 whose experts are marked in a 64-bit mask per expert, so the
// rank of an assignment among its expert's (tokens ascending) is a popcount.
// A chunk that is the whole call (up to 64 tokens) is finished here.
template <int NK, bool BF16, bool VEC>
__global__ __launch_bounds__(1024) void k_gate(GateArgs a) {
  __shared__ float xl[GATE_WAVES][NK * 64], kl[GATE_WAVES][NK * 64];
  __shared__ unsigned long long mask[GATE_MAXE];
  __shared__ int32_t run[GATE_MAXE], off[GATE_MAXE];
  __shared__ int32_t bi[64 * 16];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk;
  const int n = (int)(a.T - c0 < a.chunk ? a.T - c0 : a.chunk);
  const bool perm = a.perm != nullptr;
  float x[NK], bias[NK];
  if (wave < n) load_logits<NK, BF16, VEC>(a, c0 + wave, x);
#pragma unroll
  for (int i = 0; i < NK; ++i) bias[i] = a.bias && NK * lane + i < a.E ? a.bias[NK * lane + i] : 0.0f;
  for (int e = tid; e < a.E; e += 1024) run[e] = 0;
  for (int b0 = 0; b0 < n; b0 += 64) {
    const int nb = n - b0 < 64 ? n - b0 : 64;
    for (int e = tid; e < a.E; e += 1024) mask[e] = 0ull;
    __syncthreads();
    for (int q = wave; q < nb; q += GATE_WAVES) {
      const int64_t t = c0 + b0 + q;
      int e;
      float w, next[NK];
      // the wave's next token, while this one is worked on
      const int nq = q + GATE_WAVES < nb ? b0 + q + GATE_WAVES : b0 + 64 + wave;
      if (nq < n) load_logits<NK, BF16, VEC>(a, c0 + nq, next);
      gate_token<NK>(a, x, bias, xl[wave], kl[wave], e, w);
#pragma unroll
      for (int i = 0; i < NK; ++i) x[i] = next[i];
      if (lane < a.k) {
        if (a.idx) a.idx[t * a.k + lane] = e;
        if (a.w) a.w[t * a.k + lane] = w;
        if (perm) {
          bi[q * a.k + lane] = e;
          atomicOr(&mask[e], 1ull << q);
        }
      }
    }
    __syncthreads();
    if (!perm) continue;
    if (a.nchunk == 1) {
      for (int e = tid; e < a.E; e += 1024) {
        run[e] = __popcll(mask[e]);
        a.counts[e] = run[e];
      }
      __syncthreads();
      if (wave == 0) {
        const int all = wave_scan_512(run, off, a.E);
        if (lane == 0) a.offsets[a.E] = all;
      }
      __syncthreads();
      for (int e = tid; e < a.E; e += 1024) a.offsets[e] = off[e];
      for (int i = tid; i < nb * a.k; i += 1024) {
        const int q = i / a.k, e = bi[i];
        a.perm[off[e] + __popcll(mask[e] & ((1ull << q) - 1))] = i;
      }
      return;
    }
    for (int i = tid; i < nb * a.k; i += 1024) {
      const int q = i / a.k, e = bi[i];
      a.lrank[(c0 + b0) * a.k + i] = (uint16_t)(run[e] + __popcll(mask[e] & ((1ull << q) - 1)));
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += 1024) run[e] += __popcll(mask[e]);
    __syncthreads();
  }
  if (!perm) return;
  const int epad = (a.E + 1) & ~1;
  for (int e = tid; e < epad; e += 1024) a.ccnt[(int64_t)blockIdx.x * epad + e] = e < a.E ? (uint16_t)run[e] : 0;
}

// One workgroup per chunk: every expert's count in the chunks before this one
// and in all (a thread per two experts and every 1024 / columns-th chunk), the
// offsets, and the places of the chunk's assignments.
__global__ __launch_bounds__(1024) void k_gate_place(GateArgs a) {
  __shared__ int32_t part[2][2048];
  __shared__ int32_t before[GATE_MAXE], total[GATE_MAXE], off[GATE_MAXE];
  const int tid = threadIdx.x, b = blockIdx.x, cols = (a.E + 1) / 2;
  int wide = 32;  // threads side by side: a power of two
  while (wide < cols) wide *= 2;
  const int col = tid & (wide - 1), grp = tid / wide, ngrp = 1024 / wide;
  const uint32_t *const cc = reinterpret_cast<const uint32_t *>(a.ccnt);
  // two counts of up to 2^12 in the halves of a word: sums of at most 256 of
  // them could carry, so they are added apart
  int t0 = 0, t1 = 0, f0 = 0, f1 = 0;
  for (int c = grp; c < a.nchunk; c += 8 * ngrp) {
    uint32_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = col < cols && c + u * ngrp < a.nchunk ? cc[(c + u * ngrp) * cols + col] : 0u;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int lo = v[u] & 0xFFFF, hi = v[u] >> 16;
      t0 += lo;
      t1 += hi;
      if (c + u * ngrp < b) {
        f0 += lo;
        f1 += hi;
      }
    }
  }
  part[0][2 * tid] = t0;
  part[0][2 * tid + 1] = t1;
  part[1][2 * tid] = f0;
  part[1][2 * tid + 1] = f1;
  __syncthreads();
  for (int e = tid; e < a.E; e += 1024) {
    int t = 0, f = 0;
    for (int q = 0; q < ngrp; ++q) {
      t += part[0][2 * wide * q + e];
      f += part[1][2 * wide * q + e];
    }
    total[e] = t;
    before[e] = f;
  }
  __syncthreads();
  if (tid < 64) {
    const int all = wave_scan_512(total, off, a.E);
    if (b == 0 && tid == 0) a.offsets[a.E] = all;
  }
  __syncthreads();
  if (b == 0)
    for (int e = tid; e < a.E; e += 1024) {
      a.counts[e] = total[e];
      a.offsets[e] = off[e];
    }
  const int64_t c0 = (int64_t)b * a.chunk;
  const int n = (int)(a.T - c0 < a.chunk ? a.T - c0 : a.chunk);
  for (int i = tid; i < n * a.k; i += 1024) {
    const int64_t as = c0 * a.k + i;
    const int e = a.idx[as];
    a.perm[off[e] + before[e] + a.lrank[as]] = (int32_t)as;
  }
}

// ---------------------------------------------------------------- gradient
// One wave per token.  With w_j = scale * s_j (or scale * s_j / S):
//   d s_j = scale * dw_j                                  (weights as they come)
//   d s_j = scale / S * (dw_j - sum_i dw_i s_i / S)       (renormalised)
// and d l = ds * ds/dl; softmax without renormalisation reaches every logit:
// d l_e = p_e (ds_e - sum_j ds_j p_j).  Softmax with it is a softmax over the
// chosen logits alone.  A row is read (for the dense form) and written once:
// 8192 x 256 in fp32, 17 MB, takes 8.4 us for 3.4 us of memory: 2048 short
// workgroups of one row a wave, 4 bytes a lane and load and nothing loaded
// ahead; 1237 x 60 3.9 us.
template <int NK, bool BF16>
__global__ __launch_bounds__(256) void k_gate_backward(GateGradArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  int e = -1;
  float dw = 0.0f, l = -INFINITY;
  if (lane < a.k) {
    e = a.idx[t * a.k + lane];
    dw = a.dw[t * a.k + lane] * a.scale;
    if (e >= 0 && e < a.E && !(a.bias && !(a.bias[e] > -INFINITY)))
      l = clean_logit(load_logit<BF16>(a.logits, t * a.ld + e));
    else
      e = -1;
  }
  const bool live = l != -INFINITY;
  float g[NK];
  const bool soft = a.score == SC_SOFTMAX, dense = soft && !a.renorm;
  float mine = 0.0f;  // d l of the chosen logit
  float p[NK];
  if (dense) {
    float x[NK], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int q = lane + 64 * i;
      x[i] = q < a.E ? clean_logit(load_logit<BF16>(a.logits, t * a.ld + q)) : -INFINITY;
      m = fmaxf(m, x[i]);
    }
    m = wave_max_f(m);
    if (m == -INFINITY) m = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      p[i] = expf(x[i] - m);
      z += p[i];
    }
    z = wave_sum_f(z);
    const float zi = z > 0.0f ? 1.0f / z : 0.0f;
    const float pj = live ? expf(l - m) * zi : 0.0f;
    const float dot = wave_sum_f(live ? dw * pj : 0.0f);
#pragma unroll
    for (int i = 0; i < NK; ++i) g[i] = -p[i] * zi * dot;
    mine = live ? dw * pj : 0.0f;
  } else {
    // d s/d l * S/s: no quotient by a sum or a score that is small
    float s = 0.0f, slope = 1.0f;
    const float m = wave_max_f(l);
    if (live) {
      if (soft) s = expf(l - m);
      else s = a.renorm ? relative_score(l, a.score, m) : own_score(l, a.score);
      if (a.score == SC_SIGMOID) slope = 1.0f / (1.0f + expf(l));
      if (a.score == SC_SQRT_SOFTPLUS) {  // sigmoid / (2 softplus), below -17 the limit of that
        const float r = router_score(l);
        slope = l < -17.0f ? 0.5f : 0.5f / (r * r * (1.0f + expf(-l)));
      }
    }
    float q = s;
    const float ds = live ? dw : 0.0f;
    float dot = 0.0f;
    if (a.renorm) {
      const float S = wave_sum_f(s);
      q = S > 0.0f ? s / S : 0.0f;
      dot = wave_sum_f(ds * q);
    }
    mine = live ? (ds - dot) * q * slope : 0.0f;
#pragma unroll
    for (int i = 0; i < NK; ++i) g[i] = 0.0f;
  }
  for (int j = 0; j < a.k; ++j) {
    const int ej = __shfl(e, j);
    const float v = __shfl(mine, j);
#pragma unroll
    for (int i = 0; i < NK; ++i) g[i] += lane + 64 * i == ej ? v : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int q = lane + 64 * i;
    if (q < a.E) {
      if (BF16) ((__bf16 *)a.dl)[t * a.ldd + q] = (__bf16)g[i];
      else ((float *)a.dl)[t * a.ldd + q] = g[i];
    }
  }
}

}  // namespace

int gate_chunk(int64_t T) {
  if (T <= 64) return 64;
  int c = 16;
  while (c < 64 && (T + c - 1) / c > 256) c *= 2;
  if ((T + c - 1) / c > 256) c = (int)(((T + 255) / 256 + 63) / 64 * 64);
  return c;
}

int gate_chunks_max(int64_t T) { return T >= 4096 ? 256 : (int)((T + 15) / 16); }

hipError_t launch_gate(const GateArgs &a, hipStream_t s) {
  const dim3 g(a.nchunk), b(1024);
  // a lane's logits in one load where every row allows it
  const int nk = a.E <= 64 ? 1 : a.E <= 128 ? 2 : a.E <= 256 ? 4 : 8, size = (a.bf16 ? 2 : 4) * nk, al = size < 16 ? size : 16;
  const bool vec = nk > 1 && a.E % nk == 0 && a.ld * (a.bf16 ? 2 : 4) % al == 0 && (uintptr_t)a.logits % al == 0;
  auto run = [&](auto f32, auto f32v, auto bf, auto bfv) { hipLaunchKernelGGL(a.bf16 ? (vec ? bfv : bf) : (vec ? f32v : f32), g, b, 0, s, a); };
#define OF(NK) k_gate<NK, false, false>, k_gate<NK, false, true>, k_gate<NK, true, false>, k_gate<NK, true, true>
  if (nk == 1) run(k_gate<1, false, false>, k_gate<1, false, false>, k_gate<1, true, false>, k_gate<1, true, false>);
  else if (nk == 2) run(OF(2));
  else if (nk == 4) run(OF(4));
  else run(OF(8));
#undef OF
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.perm || a.nchunk == 1) return e;
  hipLaunchKernelGGL(k_gate_place, g, b, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateGradArgs &a, hipStream_t s) {
  const dim3 g((unsigned)(((int64_t)a.T + 3) / 4)), b(256);
  auto run = [&](auto f32, auto bf16) {
    if (a.bf16) hipLaunchKernelGGL(bf16, g, b, 0, s, a);
    else hipLaunchKernelGGL(f32, g, b, 0, s, a);
  };
  if (a.E <= 64) run(k_gate_backward<1, false>, k_gate_backward<1, true>);
  else if (a.E <= 128) run(k_gate_backward<2, false>, k_gate_backward<2, true>);
  else if (a.E <= 256) run(k_gate_backward<4, false>, k_gate_backward<4, true>);
  else run(k_gate_backward<8, false>, k_gate_backward<8, true>);
  return hipGetLastError();
}

}  // namespace ds4
