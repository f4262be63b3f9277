// spa_latent_ring.h - positions in the rings of buffers and barriers of the latent kernels.  Plain C++
// with no CUDA dependency, so that the order of the kernels' waits can be checked on a machine without
// a GPU (tests/latent_order.cpp walks every interleaving of their warps with these rings).
//
// A wait by parity tells the phase it is for from the phases just before and just after it, and from
// no other.  So it is sound only if, whenever a warp comes to it, that phase is either the next to be
// completed or the last that was.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SPA_HOST_DEVICE __host__ __device__
#else
#define SPA_HOST_DEVICE
#endif

namespace spa {

// Use k of a ring of N is at slot k % N, and is phase k / N of that slot's barriers.
template <int N>
struct Ring {
  static constexpr int kSlots = N;
  int slot = 0;
  uint32_t parity = 0;    // of the phase
  SPA_HOST_DEVICE void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// Tiles of rows in the decode kernel's shared memory: a tile's FULL, EMPTY and P-ready barriers are all
// at its slot of this ring.
using LatentTileRing = Ring<3>;

}  // namespace spa
