// How the tile kernels of the packed products share out their work: tiles of the
// output over as many workgroups as the card holds at once, the last ones split over
// the contraction.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dma_common.hpp"

namespace dora {

constexpr int kCUs = 256;

struct TileGrid {
  int S;  // stages of the contraction
  // units of work: tiles [0, whole) over the whole contraction, then tiles
  // [whole, nRB * nTiles) in nSplit ranges of its stages each
  int nRB, nTiles, whole, nSplit;
  uint32_t group;  // column tiles of a group of the tile order
};

// Tile order: groups of `group` column tiles, row blocks within a group, on
// XCD-contiguous ranges: an XCD's concurrent tiles form a block of rows and
// columns whose panels its L2 holds for all of them.
__device__ inline void tile_of(uint32_t v, const TileGrid& a, int& rb, int& nt) {
  const uint32_t nRB = static_cast<uint32_t>(a.nRB), nTl = static_cast<uint32_t>(a.nTiles), G = a.group;
  const uint32_t grp = v / (G * nRB);
  const uint32_t gn = min(G, nTl - grp * G);
  const uint32_t loc = v - grp * G * nRB;
  rb = static_cast<int>(loc / gn);
  nt = static_cast<int>(grp * G + loc % gn);
}

// The k-th unit of work of this workgroup (of the 8 XCDs x gridDim.x/8): false
// past its last.  An XCD takes contiguous ranges of the whole tiles and of the
// split ones.
struct Unit {
  int rb, nt, st0, st1, split, tail;  // tail: index among the split tiles, -1 for a whole tile
};
__device__ inline bool unit_of(int k, const TileGrid& a, Unit& u) {
  // (opaque, so that nothing of this moves out of the rare branches it stands in)
  asm volatile("" : "+s"(k));
  const int x = blockIdx.x & 7, i = blockIdx.x >> 3, per = gridDim.x >> 3;
  const int wpx = (a.whole + 7) >> 3;  // whole tiles of an XCD
  const int w0 = min(x * wpx, a.whole), w1 = min(w0 + wpx, a.whole);
  const int rounds = (w1 - w0 + per - 1 - i) / per;  // whole tiles of this workgroup
  int v;
  if (k < rounds) {
    v = w0 + k * per + i;
    u.st0 = 0;
    u.st1 = a.S;
    u.split = 0;
    u.tail = -1;
  } else {
    const int ntail = a.nRB * a.nTiles - a.whole, nun = ntail * a.nSplit, upx = (nun + 7) >> 3;
    const int j = (k - rounds) * per + i, n = x * upx + j;
    if (j >= upx || n >= nun) return false;
    u.split = n / ntail;
    u.tail = n - u.split * ntail;
    v = a.whole + u.tail;
    u.st0 = a.S * u.split / a.nSplit;  // S <= 2^16
    u.st1 = a.S * (u.split + 1) / a.nSplit;
  }
  tile_of(static_cast<uint32_t>(v), a, u.rb, u.nt);
  return true;
}

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                           kBufferWord3);
}

}  // namespace dora
