// Addressing inside a paged 4-bit key/value cache (layout: mnb.h, "Paged 4-bit key/value cache").
#pragma once

#include <stdint.h>

namespace mnb {
namespace kv4 {

// Byte of K word (t, w) of row r: the words that one lane of the QK product reads (one t, every w) are
// contiguous, and eight lanes of two rows cover all 32 banks (D = 256: through the swap of
// the two 16-byte halves in odd rows).
template <int D>
__host__ __device__ constexpr int k_word_byte(int r, int t, int w) {
  return r * (D / 2) + (t * (D / 32) + (w ^ (D == 256 ? (r & 1) * 4 : 0))) * 4;
}

// Place of row r in chunk g of the V codes, which spreads the chunks of the PV product's
// lanes over the banks.
template <int D>
__host__ __device__ constexpr int v_place(int r, int g) {
  return r ^ (D == 64 ? ((g >> 1) & 1) * 8 : D == 128 ? (g & 1) * 8 : (g & 1));
}

// Byte of V word (g, r, w), from the start of the V codes.
template <int D>
__host__ __device__ constexpr int v_word_byte(int g, int r, int w) {
  return (g * 16 + v_place<D>(r, g)) * (D / 16) + w * 4;
}

// Byte of 16-byte chunk `chunk` of row `row` (of 128) in the tcgen05 kernel's shared memory of one row tile: 64 fp16
// elements of a row are 128 bytes, swizzled, and the next 64 follow after those of all rows. q lies so, and
// results pass through the same places on their way out: a row's bytes belong to its own warp from the
// start of a piece to its end, so the warps need no barrier between one piece's results and the next one's q.
__host__ __device__ constexpr int tile_row_byte(int row, int chunk) {
  return (chunk >> 3) * (128 * 128) + row * 128 + ((chunk ^ row) & 7) * 16;
}

}  // namespace kv4
}  // namespace mnb
