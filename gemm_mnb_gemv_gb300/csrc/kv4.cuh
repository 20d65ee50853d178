// Addressing inside a paged 4-bit key/value cache (layout: mnb.h, "Paged 4-bit key/value cache").
#pragma once

#include <cuda_fp16.h>
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

}  // namespace kv4
}  // namespace mnb
