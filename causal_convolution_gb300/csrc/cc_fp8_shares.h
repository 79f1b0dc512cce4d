// How the 8-bit product divides the blocks of K among the CTA pairs of a
// cluster. Plain C++, so that the host can sweep it.
#pragma once

#ifdef __CUDACC__
#define CC_HOST_DEVICE __host__ __device__
#else
#define CC_HOST_DEVICE
#endif

namespace cc {

// Blocks of K of every pair but the last ones, whose shares may be shorter or
// empty: whole fours, because the scales come in fours.
CC_HOST_DEVICE constexpr int share_blocks(int kblocks, int pairs) { return ((kblocks - 1) / pairs + 4) / 4 * 4; }

// Blocks of the pair whose share begins at block `first`. With none, rows end at
// or in front of `first`.
CC_HOST_DEVICE constexpr int blocks_in_share(int kblocks, int share, int first) {
  return first >= kblocks ? 0 : kblocks - first < share ? kblocks - first : share;
}

// The block from which on a pair asks for its first four scales.
CC_HOST_DEVICE constexpr int first_request(int blocks, int first) { return blocks > 0 ? first : 0; }

}  // namespace cc
