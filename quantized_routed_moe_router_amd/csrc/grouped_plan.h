// Which instance of the tiled kernels takes a product grouped by expert, or a
// gradient of one, and the workgroups of its launch: arithmetic of the host
// alone, without the runtime's headers.
#pragma once
#include <stdint.h>

namespace ds4 {

// waves of a workgroup (32 columns of the result each) and the height of its
// tiles in rows, 0 for one that the kernel chooses by the numbers of rows
struct GroupedForm {
  int waves, height;
  int64_t lowest() const { return height ? height : waves == 8 ? 128 : 64; }  // that the kernel may choose
  int64_t columns() const { return 32 * waves; }
};

// the most tiles of `height` rows or more that the segments of P rows can make:
// one of all rows, or E experts' and the two of no expert
inline int64_t grouped_max_tiles(bool ragged, int64_t E, int64_t P, int64_t height) {
  return ragged ? P / height + (P < E + 2 ? P : E + 2) : (P + height - 1) / height;
}
inline int64_t grouped_col_tiles(GroupedForm f, int64_t N) { return (N + f.columns() - 1) / f.columns(); }
inline int64_t grouped_workgroups(GroupedForm f, bool ragged, int64_t E, int64_t P, int64_t N) {
  return (grouped_max_tiles(ragged, E, P, f.lowest()) * grouped_col_tiles(f, N) + 7) / 8 * 8;
}

// All rules go by sizes alone: how many rows each expert has is known on the
// device only.  Times are calls in us on one MI355X, of bf16 matrices of 2048 x
// 4096 where nothing else is said, with experts drawn evenly; "skewed" is by a
// power of -1.1 of their rank.

// Few rows: a kernel whose workgroups have 16 rows of weights and 16 of x
// against tiles of up to 64 rows.  256 experts: 64 rows in all 160 and 164, 256
// 512 and 533, 512 677 and 709, 1024 823 and 822, 2048 978 and 776.  8 experts:
// 4 rows 9 and 26, 16 20 and 26, 32 27 and 29, 128 42 and 30.  Of one matrix (8
// bits, where it takes up to 64 rows at once): 16 rows 7.7 and 15, 64 13 and
// 16; of 8192 x 4096 32 rows 14.7 and 15.2, 64 23 and 16.
// Up to 2 E it loses where few experts have the rows, whose weights it reads
// once per 16: 256 rows of 256 experts skewed 330 and 264, all of one expert
// 152 and 28; and of 8 bits: 256 rows of 256 experts 329 and 236, 16 of 8 17.6
// and 16.4 (8 of 8 13 and 16).
inline bool grouped_is_few(bool ragged, int64_t E, int64_t P) { return ragged ? P <= 2 * E : P <= 64; }

// More rows: eight waves or four, by the number of results.  Up to 128 rows an
// expert (64) the tiles are as high as that, so that its weights are read once;
// beyond, the kernel chooses.  The bound stands between measured sizes, where
// the sides cross.  Eight and four, both with the choice, by millions of
// results: 8 experts 16.8 112 and 125, 18.9 148 and 144, 23.1 176 and 172, 25.2
// 189 and 179, 27.3 208 and 225, 33.5 228 and 269; skewed (-0.6) 141 and 138,
// 145 and 145, 178 and 168, 191 and 214, 213 and 221, 281 and 276.  4 experts of
// 8192 x 4096: 21.0 184 and 180, 25.2 195 and 195, 29.4 210 and 267.  8 bits, 8
// experts: 23.1 106 and 105, 25.2 109 and 108, 27.3 124 and 131.
// Eight of 128 rows and four of 64: 128 experts 25.2 397 and 536 (skewed 510 and
// 592); 256 of 1024 x 1024 25.2 139 and 146 (149 and 159); 8 bits 233 and 274, 101
// and 111.  Below, 64 rows each: 8 experts 38 and 28, 16 55 and 44, 256 of 1024 x
// 1024 124 and 119 - but 64 experts 188 and 242, and 128 experts 377 and 499 (8
// bits 133 and 124, 212 and 229): there the tiles of all weights, E N / 256, would
// tell the sides apart better than the results do.
constexpr int64_t kEightWaves = 24000000;
inline GroupedForm grouped_form(bool ragged, int64_t E, int64_t P, int64_t N) {
  const int64_t mean = ragged ? P / E : P;  // rows of an expert
  if (P * N >= kEightWaves) return mean <= 128 ? GroupedForm{8, 128} : GroupedForm{8, 0};
  return mean <= 64 ? GroupedForm{4, 64} : GroupedForm{4, 0};
}
// Turned weights, fp32 results: of 256 experts 64 rows each eight waves 857 and
// four 943, 16 rows each 774 and 830; with matrices of 1024 x 1024 145 and 143,
// 16 rows each 110 and 110; 512 experts of 264 x 264, 64 rows each, 61 and 54.
// Below: 60 experts (488 x 1000) 62 rows each 21.7 and 19.7, 128 of 512 x 1024
// 64 rows each 47 and 42, 8 experts 128 rows each 42 and 37.  Many rows, eight
// waves of 128 rows and four with the choice: 8 experts 512 rows each 94 and 93
// (skewed 122 and 100), 1024 188 and 188 (210 and 188).
// Beyond 2^35 results (64 GiB of 16 bits) it is eight waves again, whose tiles
// are four times as large: four waves' could be 2^24, with more threads than a
// launch has, and the sizes that the kernel compares would leave 32 bits.
inline GroupedForm grouped_turned_form(int64_t E, int64_t P, int64_t N) {
  const int64_t mean = P / E;
  if (P * N > (int64_t)1 << 35 || (mean <= 128 && E * ((N + 255) / 256) >= 1024)) return {8, 128};
  return mean <= 64 ? GroupedForm{4, 64} : GroupedForm{4, 0};
}

// The gradient of the weights: tiles of 256 x 256 (one workgroup on a CU) or
// 128 x 128 (three), by the number of the large ones; the bound stands between
// measured numbers.  32768, 64 terms each, 1170 and 1288; 4096 of 256 experts of
// 1024 x 1024, 64 terms, 152 and 185 (skewed 235 and 270); 2048 of 16 experts, 64
// terms, 66 and 71 (93 and 108), 512 terms 161 and 193 (329 and 310); 1536 of 96
// of 1024 x 1024, 256 terms, 93 and 112 (183 and 166).  1024, 1024 terms each,
// within a whole backward pass: of 8 experts 345 and 358, of 64 of 1024 x 1024
// 450 and 483.  960 of 60 experts, 62 terms each, 36 and 30; 480 44 and 38; 128,
// 4096 terms, 115 and 73.
// Few terms make the small ones the better at higher numbers too: 1536 of 12
// experts, 64 terms, 50 and 46 (72 and 66); 1024 of 256 of 512 x 512 38 and 32
// (101 and 60); and large tiles that are mostly empty at any: 2048 of 512 experts
// of 264 x 264 59 and 30.
constexpr int64_t kLargeTiles = 1000;
inline bool grouped_dw_large(int64_t E, int64_t N, int64_t K) { return E * ((N + 255) / 256) * ((K + 255) / 256) >= kLargeTiles; }
inline int64_t grouped_dw_workgroups(bool large, int64_t E, int64_t N, int64_t K) {
  const int64_t side = large ? 256 : 128;
  return (E * ((N + side - 1) / side) * ((K + side - 1) / side) + 7) / 8 * 8;
}

}  // namespace ds4
