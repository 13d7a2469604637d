// Counter-based random words for dropout: Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011).  Ten rounds of
//   (x0, x1, x2, x3) <- (hi(m1 x2) ^ x1 ^ k0, lo(m1 x2), hi(m0 x0) ^ x3 ^ k1, lo(m0 x0)),
// the key advancing by two Weyl constants a round, turn a 128-bit counter into
// four independent 32-bit words.  Element e of a row-major tensor takes word e & 3
// of the counter (e >> 2, offset) under the key `seed`, so forward and backward
// form the same mask from two numbers and no mask is stored.
#pragma once

#include <stdint.h>

#include "kernels.h"

namespace qlora {

// The round keys come with the launch (they depend on the seed alone), so a round is
// two wide products and two three-way exclusive ors.
__device__ __forceinline__ uint4 philox4x32_10(uint64_t block, uint64_t offset, const DropoutCounter& d) {
  uint32_t x0 = static_cast<uint32_t>(block), x1 = static_cast<uint32_t>(block >> 32);
  uint32_t x2 = static_cast<uint32_t>(offset), x3 = static_cast<uint32_t>(offset >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * x0, b = static_cast<uint64_t>(0xCD9E8D57u) * x2;
    x0 = static_cast<uint32_t>(b >> 32) ^ x1 ^ d.key[2 * i];
    x2 = static_cast<uint32_t>(a >> 32) ^ x3 ^ d.key[2 * i + 1];
    x1 = static_cast<uint32_t>(b);
    x3 = static_cast<uint32_t>(a);
  }
  return make_uint4(x0, x1, x2, x3);
}

// The offset of one launch: the host's value plus the device counter, if any.
__device__ __forceinline__ uint64_t dropout_offset(const DropoutCounter& d) {
  return d.offset + (d.counter ? *d.counter : 0ull);
}

}  // namespace qlora
