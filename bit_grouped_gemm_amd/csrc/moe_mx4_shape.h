// moe_mx4_shape.h -- which kernel and tile a row-major MXFP4 product takes, by
// its sizes (host code only, without HIP).
#pragma once

#include <cmath>

namespace moe {

constexpr int kMx4Cols = 256;  // columns of k_mx4's tiles

// The shape of a launch: rows and columns of a tile, and the kernel that makes it.
enum { kMx4Big, kMx4Few, kMx4Rows };  // k_mx4; k_mx4_few with WK = 4; with WK = 1
struct Mx4Shape {
  int kind, rows, cols;
};

// The shape that is expected to take the least time.  A launch takes a start and its rounds
// of as many tiles as the CUs hold; a round what a tile takes by itself (its
// turn, and its K steps one after the other) or what its bytes take through a CU,
// whichever is more.  The numbers, in us, are fitted to the 17 shapes' times on 33 products
// (1 to 32768 rows in 1 to 128 groups, K 256 to 16384, N 128 to 7168): the shape that
// is chosen is the fastest of them in 31, and 3 % slower in two.
//   us, fastest and others: one row, 7168 -> 4096: Few 16 x 16 7.0, 16 x 64 12.9; 600 rows, 4096 ->
//   4096: Big 128 18.8, 256 27.6, Few 64 x 64 25.8, Rows 64 x 128 29.5; top-8 of 64: 61
//   tokens, 2048 -> 7168: Rows 16 x 128 86.8, Big 128 109.5; 512 tokens, 4096 -> 1536: Big 128
//   56.7, 256 64.9, Rows 32 x 256 85.3; 4096 tokens: Big 256 145, 128 176.  (Of one process each; from process
//   to process all of a product's times move together, by up to 15 %.)
// The row tiles of ragged groups are estimated: groups with a row, each half a tile more
// than its mean needs.
inline Mx4Shape mx4_shape(int R, int N, int K, int E, double* cost_of = nullptr) {
  constexpr double kCUs = 256;
  struct Cost {
    double start, turn, step, rate;  // us, us, us per step of a wave, bytes per us and CU
  };
  static const Cost cost_of_kind[] = {{0, 11, 0.85, 35e3}, {5, 0.8, 1.05, 31e3}, {0.4, 2.8, 0.72, 40e3}};
  struct Shape {
    Mx4Shape s;
    int share;  // workgroups that a CU holds
  };
  static const Shape shapes[] = {
      {{kMx4Few, 16, 16}, 2},        {{kMx4Few, 16, 32}, 2},         {{kMx4Few, 16, 64}, 1},
      {{kMx4Few, 32, 16}, 2},        {{kMx4Few, 32, 32}, 2},         {{kMx4Few, 32, 64}, 1},
      {{kMx4Few, 64, 16}, 1},        {{kMx4Few, 64, 32}, 1},         {{kMx4Few, 64, 64}, 1},
      {{kMx4Rows, 16, 64}, 4},       {{kMx4Rows, 16, 128}, 2},       {{kMx4Rows, 16, 256}, 1},
      {{kMx4Rows, 32, 128}, 2},      {{kMx4Rows, 32, 256}, 1},       {{kMx4Rows, 64, 128}, 1},
      {{kMx4Big, 128, kMx4Cols}, 1}, {{kMx4Big, 256, kMx4Cols}, 1}};
  const double groups = E * (1.0 - std::exp(-double(R) / E));  // that are touched
  const double mean = R / std::fmax(groups, 1.0), bytes = K / 2.0 + K / 32.0;
  Mx4Shape best = {kMx4Big, 256, kMx4Cols};
  double least = 1e300;
  for (const Shape& shape : shapes) {
    const Mx4Shape& s = shape.s;
    const Cost& c = cost_of_kind[s.kind];
    const double rows = E == 1 ? std::ceil(R / double(s.rows)) : groups * std::fmax(1.0, mean / s.rows + 0.5);
    const double tiles = std::ceil(rows) * std::ceil(double(N) / s.cols);
    const double rounds = std::ceil(tiles / (kCUs * shape.share));
    // (a step of the large tiles takes as long as they have rows, and a bit; the others' four
    // waves have a quarter of the steps each, or all)
    const double steps = std::ceil(K / 256.0) * (s.kind == kMx4Big ? s.rows / 256.0 + 0.3 : s.kind == kMx4Few ? 0.25 : 1.0);
    const double turns = s.kind == kMx4Big ? rounds : tiles / kCUs;
    const double cost =
        c.start + std::fmax(rounds * (c.turn + steps * c.step), turns * (s.rows + s.cols) * bytes / c.rate);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  if (cost_of) *cost_of = least;
  return best;
}

// Rows of a dense product's first launch.  Where the last few rows would make the
// large tiles go one more round, they go into a launch of their own, in the shape
// that suits them, if that is expected to save the time of a launch.
inline int mx4_first_rows(int R, int N, int K) {
  constexpr double kLaunchTime = 5;
  const int rows = R / 256 * 256;
  if (R <= 256 || rows == R) return R;
  double one, head, tail;
  mx4_shape(R, N, K, 1, &one);
  mx4_shape(rows, N, K, 1, &head);
  mx4_shape(R - rows, N, K, 1, &tail);
  return head + tail + kLaunchTime < one ? rows : R;
}

}  // namespace moe
