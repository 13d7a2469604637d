// The keep mask of the counter-based dropout written out as bytes, for callers
// that keep masks (and to check the kernels that never store one).  One thread
// forms 16 elements (four Philox blocks) and writes them with one 16-byte store.  A
// round is two wide products and two exclusive ors, so ten rounds and the comparisons
// are about 12 integer instructions an element against one byte written: bound by
// those, not by memory (8192 x 4096 27 us, 1.24 TB/s; 2^30 elements 814 us, 1.32 TB/s).
#include "common.cuh"
#include "kernels.h"
#include "philox.cuh"

namespace qlora {

namespace {

constexpr int kDmThreads = 256;

__global__ void __launch_bounds__(kDmThreads) dropout_mask_kernel(const __grid_constant__ DropoutCounter d, int64_t n, uint8_t* keep) {
  const int64_t e0 = (static_cast<int64_t>(blockIdx.x) * kDmThreads + threadIdx.x) * 16;
  if (e0 >= n) return;
  const uint64_t off = dropout_offset(d);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 u = philox4x32_10(static_cast<uint64_t>(e0 / 4 + i), off, d);
    w[i] = (u.x >= d.threshold ? 1u : 0u) | (u.y >= d.threshold ? 0x100u : 0u) |
           (u.z >= d.threshold ? 0x10000u : 0u) | (u.w >= d.threshold ? 0x1000000u : 0u);
  }
  if (n - e0 >= 16) {
    *reinterpret_cast<uint4*>(keep + e0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    for (int i = 0; i < n - e0; ++i) keep[e0 + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

}  // namespace

void philox_keys(uint64_t seed, uint32_t (&key)[20]) {
  for (uint32_t i = 0; i < 10; ++i) {
    key[2 * i] = static_cast<uint32_t>(seed) + i * 0x9E3779B9u;
    key[2 * i + 1] = static_cast<uint32_t>(seed >> 32) + i * 0xBB67AE85u;
  }
}

cudaError_t launch_dropout_mask(const DropoutCounter& d, int64_t n, uint8_t* keep, cudaStream_t stream) {
  const int64_t grid = (n + kDmThreads * 16 - 1) / (kDmThreads * 16);
  dropout_mask_kernel<<<static_cast<unsigned>(grid), kDmThreads, 0, stream>>>(d, n, keep);
  count_launch();
  return cudaGetLastError();
}

}  // namespace qlora
