// How the adapters' kernels share out their work: the list of (column block, row
// tile), row tiles of up to 128 positions in group order, is cut into equal runs
// for the CTAs, so that the groups' sizes do not unbalance it.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace e4b {

constexpr int kTile = 128;  // positions of a row tile, at most

// Positions of a row tile: 128, or another power of two.
struct FullTile {
  __host__ __device__ int shift() const { return 7; }
};
struct AnyTile {
  int bits;
  __host__ __device__ int shift() const { return bits; }
};

template <typename Size>
__host__ __device__ inline int64_t group_tiles(const int64_t* offsets, int g, int64_t R_max, int64_t& beg, int64_t& end,
                                               Size size) {
  beg = offsets[g];
  end = offsets[g + 1];
  beg = beg < 0 ? 0 : beg > R_max ? R_max : beg;  // no position outside [0, R_max) is ever formed
  end = end < 0 ? 0 : end > R_max ? R_max : end;
  return end > beg ? (end - beg + (1 << size.shift()) - 1) >> size.shift() : 0;
}

// a / b for a >= 0, b > 0, in 32 bits where they fit: a kernel's start waits for
// these divisions (in 64 bits they took a microsecond).
E4B_DEV int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// A CTA's run: the column block it begins in, and its items.
struct Run {
  int block;
  int64_t count;
};

// By the whole CTA (ends with a barrier): the row tiles of all groups are added
// up, and start receives the group and the tile within it that the run begins
// with. sums: [THREADS / 32]. count 0: nothing is left for this CTA.
template <int THREADS, typename Size>
E4B_DEV Run find_run(const int64_t* __restrict__ offsets, int G, int64_t R_max, int blocks, Size size, int64_t* sums,
                     int64_t* start) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int strip = (G + THREADS - 1) / THREADS;
  const int lo = min(tid * strip, G), hi = min(lo + strip, G);
  int64_t beg, end, mine = 0;
  for (int g = lo; g < hi; ++g) mine += group_tiles(offsets, g, R_max, beg, end, size);
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, T = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += sums[w];
    T += sums[w];
  }
  const int64_t W = T * blocks, b = blockIdx.x;
  if (b >= W) return Run{0, 0};  // uniform; also where no group has rows
  // the first `longer` runs have an item more
  const int64_t length = quotient(W, gridDim.x), longer = W - length * gridDim.x;
  const int64_t w0 = b * length + min(b, longer), count = length + (b < longer);
  const int block = int(quotient(w0, T));
  const int64_t first = w0 - block * T;
  if (first >= before && first < before + mine) {
    int64_t left = first - before;
    for (int g = lo; g < hi; ++g) {
      const int64_t t = group_tiles(offsets, g, R_max, beg, end, size);
      if (left < t) {
        start[0] = g;
        start[1] = left;
        break;
      }
      left -= t;
    }
  }
  __syncthreads();
  return Run{block, count};
}

// A position in the list of (column block, row tile), row tiles in group order.
template <typename Size>
struct Walk {
  const int64_t* offsets;
  int64_t R_max, beg, end, tiles;
  int64_t tile;  // within the group
  int G, g, cb;
  Size size;

  E4B_DEV Walk(const int64_t* offs, int groups, int64_t r_max, const Run& run, Size tile_size, const int64_t* start)
      : offsets(offs), R_max(r_max), tile(start[1]), G(groups), cb(run.block), size(tile_size) {
    enter(int(start[0]));
  }
  E4B_DEV void enter(int group) {
    g = group;
    tiles = group_tiles(offsets, g, R_max, beg, end, size);
  }
  E4B_DEV void next() {
    if (++tile < tiles) return;
    tile = 0;
    do {
      if (g + 1 == G) ++cb;
      enter(g + 1 == G ? 0 : g + 1);
    } while (tiles == 0);  // some group has rows
  }
  E4B_DEV bool first() const { return tile == 0; }
  E4B_DEV bool last() const { return tile + 1 == tiles; }
  E4B_DEV int64_t row0() const { return beg + (tile << size.shift()); }
  E4B_DEV int n() const { return int(min(end - row0(), int64_t(1) << size.shift())); }
};

}  // namespace e4b
