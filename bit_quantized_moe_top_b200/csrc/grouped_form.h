// Which form of the grouped products' kernel a call takes: plain host code, so
// that tests can look at every choice without a GPU.
#pragma once
#include <algorithm>

#ifdef __CUDACC__
#define MOEQ_HOST_DEVICE __host__ __device__
#else
#define MOEQ_HOST_DEVICE
#endif

namespace moeq {

// CTAs per tile (1, or a pair), rows per tile at most, CTAs that split K (cg = 1)
struct ProductForm {
  int cg, width, S;
};

// Tile width and form, by an estimate of cycles. Groups are taken as equally
// large (their sizes are only known on the device). Per 128 bytes of K a CTA
// needs the larger of its MMAs, 2 cycles a row, and its L2 reads of 128
// channels and the rows it copies, at 60 bytes a cycle or its share of 6600 of
// all (8192 x 4096 x 4096 reads 12.5 TB/s). So narrower tiles cost nearly as
// much as wide ones, and it is the number of tiles that a CTA works off one
// after the other that counts. The split of K (CG = 1) pays an exchange of the
// partial sums, about 1500 cycles and 55 a column, a pair about 300 to set up.
// Clusters of eight are left out: not all of those that would fill the SMs find
// room at once (1 x 7168 x 2048 17.0 us, four 10.6). Over 38 sizes of 1 to 2000
// rows the choice took at most 10% more than the best of all forms, 2% on average.
// kBytes: of a row of K.
inline ProductForm choose_form(int rows, int E, int N, long long kBytes, int sms) {
  constexpr int kRow = 128, kBox = 32;  // bytes of K per stage, rows per copy of x
  const int nk = (int)((kBytes + kRow - 1) / kRow), pairs = sms / 2;
  const int groups = std::min(rows, E), mean = (rows - 1) / groups + 1;
  const int nf[3] = {0, (N - 1) / 128 + 1, (N - 1) / 256 + 1};  // channel tiles by CG
  const double streamed = (double)groups * N * nk * (kRow / 3500.0);  // weights at HBM's bytes per cycle
  auto cost_of = [&](const ProductForm& f) {
    const int nt = (mean - 1) / f.width + 1, unit = 16 * f.cg;
    const int n = ((mean - 1) / nt / unit + 1) * unit;
    const int tiles = groups * nt * nf[f.cg], slots = f.cg == 2 ? pairs : sms / f.S, waves = (tiles - 1) / slots + 1;
    const double rate = std::min(60.0, 6600.0 / (f.cg * f.S * std::min(tiles, slots)));
    const int loaded = (n / f.cg + kBox - 1) / kBox * kBox;
    const double per_k = std::max(2.0 * n, (128 + loaded) * kRow / rate) + 0.1 * n;  // fewer MMAs where reads bound both
    return std::max(waves * per_k * ((nk - 1) / f.S + 1), streamed) + (f.S > 1 ? 1500 + 55 * n : 0) + (f.cg == 2 ? 300 : 0);
  };
  ProductForm best{2, 256, 1};
  double least = cost_of(best);
  auto consider = [&](ProductForm f) {
    const double cost = cost_of(f);
    if (cost < least) {
      least = cost;
      best = f;
    }
  };
  for (int w = 224; w >= 64; w -= 32)
    if (mean > w - 32) consider({2, w, 1});  // a narrower tile holds the rest
  // few tiles: single CTAs, split along K while there are CTAs for it
  for (int w = 128; w >= 16; w /= 2) {
    if (mean <= w / 2 && w > 16) continue;
    const int tiles = groups * nf[1] * ((mean - 1) / w + 1);
    for (int s = 1; s <= 4 && tiles * s <= sms; s *= 2)
      if (s == 1 || nk >= s * 2) consider({1, w, s});
  }
  return best;
}

// The tiles of the last, incomplete turn of the persistent pairs go to two or
// four of them each, by rows, where that many are free: half a tile takes about
// three quarters of its time (4095 x 7168 x 4096, 256 tiles on 74 pairs, 8-bit
// 80 -> 75 us; 9000 x 4096 x 1792 in 4 experts, 16-bit 99 -> 95 us).
MOEQ_HOST_DEVICE inline int last_turn_parts(int rest, int clusters) {
  return rest * 4 <= clusters ? 4 : rest * 2 <= clusters ? 2 : 1;
}

}  // namespace moeq
