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

// few rows: a kernel whose workgroups have 16 rows of the result's columns
inline bool grouped_is_few(bool ragged, int64_t E, int64_t P) { return ragged ? P <= 2 * E : P <= 64; }

// Rules, with times in us on one MI355X of bf16 matrices of 2048 x 4096.
// Few rows an expert: tiles as high as those, so that its weights are read
// once.  64 rows each: of 256 experts eight waves 782 at a height of 128 and
// 920 at 64 (four waves 822), of 8 experts four waves 28 at 64, 43 at 128, 30
// with the choice (eight 39); 128 rows each of 8 experts 45 at 64, 48 at 128.
// Many rows: 2048 each of 8 experts 248 by eight waves with the choice and 256
// by four, 1024 each 154 and 152, 256 each 60 and 56.
inline GroupedForm grouped_form(bool ragged, int64_t E, int64_t P, int64_t N) {
  const int64_t mean = ragged ? P / E : P;  // rows of an expert
  if (P * N >= (1 << 25)) return mean <= 128 ? GroupedForm{8, 128} : GroupedForm{8, 0};
  return mean <= 64 ? GroupedForm{4, 64} : GroupedForm{4, 0};
}
// Turned weights, fp32 results: of 256 experts 64 rows each eight waves 857 and
// four 943, 16 rows each 774 and 830, of 60 experts (488 x 1000) 62 rows each
// 21.7 and 19.7; of 8 experts 1024 rows each eight waves with the choice 149 to
// 165 and four 149, 2048 rows each 290 and 271.
// Beyond 2^35 results (64 GiB of 16 bits) it is eight waves again, whose tiles
// are four times as large: four waves' could be 2^24, with more threads than a
// launch has, and the sizes that the kernel compares would leave 32 bits.
inline GroupedForm grouped_turned_form(int64_t E, int64_t P, int64_t N) {
  const int64_t mean = P / E;
  if (P * N > (int64_t)1 << 35 || (mean <= 128 && E * ((N + 255) / 256) >= 1024)) return {8, 128};
  return mean <= 64 ? GroupedForm{4, 64} : GroupedForm{4, 0};
}

// The gradient of the weights: tiles of 256 x 256 (one workgroup on a CU) or
// 128 x 128 (three).  32768 of the large ones, 64 terms each, 1170 us and 1288;
// 1024, 1024 terms each, 155 and 158; 480, 62 terms each, 44 and 38; 128, 4096
// terms each, 115 and 73.
inline bool grouped_dw_large(int64_t E, int64_t N, int64_t K) { return E * ((N + 255) / 256) * ((K + 255) / 256) >= 1024; }
inline int64_t grouped_dw_workgroups(bool large, int64_t E, int64_t N, int64_t K) {
  const int64_t side = large ? 256 : 128;
  return (E * ((N + side - 1) / side) * ((K + side - 1) / side) + 7) / 8 * 8;
}

}  // namespace ds4
