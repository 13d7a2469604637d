// A few tokens (M <= 16) through a weight of 4-bit integers with one scale per 16:
//
//   Y[m][n] = sum_k x[m][k] q[k][n] s[k][n / 16] + sum_j V[m][j] B[j][n]
//
// bound by reading the codes and scales once (0.75 B a weight).  A CTA takes 64
// columns and all rows: thread (w, l) multiplies the 8 columns of one 32-bit code
// word by the rows l, l + 32, ..., four tokens at a time, and the 32 row lanes are
// added through shared memory in a fixed order.
#include "common.cuh"
#include "kernels.h"

namespace qlora {

namespace {

constexpr int kMvThreads = 256;
constexpr int kMvTok = 4;

struct MvArgs {
  const uint32_t* codes;
  const float* scales;
  const void* x;
  const float* x_scales;
  int x_block;
  const uint16_t* V;
  const uint16_t* B;
  int M, r;
  int64_t K, N;
  uint16_t* Y;
};

__global__ void __launch_bounds__(kMvThreads) matvec_kernel(const MvArgs p) {
  __shared__ float red[32][kMvTok][64];
  const int w = threadIdx.x & 7, l = threadIdx.x >> 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64 + 8 * w;
  const int m0 = blockIdx.y * kMvTok;
  float acc[kMvTok][8] = {};
  for (int64_t k = l; k < p.K; k += 32) {
    const uint32_t c = p.codes[(k * p.N + n0) / 8];
    const float s = p.scales[(k * p.N + n0) / 16];
    float wv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wv[j] = s * static_cast<float>(static_cast<int>((c >> (4 * j)) & 15u) - 8);
#pragma unroll
    for (int t = 0; t < kMvTok; ++t) {
      const int m = m0 + t;
      if (m >= p.M) break;
      float x;
      if (p.x_scales)
        x = mul_rn(e4m3_to_float(static_cast<const uint8_t*>(p.x)[m * p.K + k]),
                   p.x_scales[p.x_block ? m * (p.K / 64) + k / 64 : m]);
      else
        x = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.x)[m * p.K + k]) << 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t][j] = fmaf(x, wv[j], acc[t][j]);
    }
  }
#pragma unroll
  for (int t = 0; t < kMvTok; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) red[l][t][8 * w + j] = acc[t][j];
  __syncthreads();
  const int t = threadIdx.x >> 6, col = threadIdx.x & 63, m = m0 + t;
  if (m >= p.M) return;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + col;
  float y = 0.0f;
  for (int i = 0; i < 32; ++i) y += red[i][t][col];
  for (int j = 0; j < p.r; ++j)
    y = fmaf(__uint_as_float(static_cast<uint32_t>(p.V[m * p.r + j]) << 16),
             __uint_as_float(static_cast<uint32_t>(p.B[j * p.N + n]) << 16), y);
  p.Y[m * p.N + n] = static_cast<uint16_t>(pack_bf16x2(y, 0.0f));
}

}  // namespace

cudaError_t launch_matvec(const WeightView& w, const ActView& x, const uint16_t* V, const uint16_t* B, int64_t M,
                          int r, uint16_t* Y, uint32_t* status, cudaStream_t stream) {
  (void)status;
  const MvArgs a{reinterpret_cast<const uint32_t*>(w.codes), w.dq_scales, x.x, x.scales, x.block, V, B,
                 static_cast<int>(M), r, w.in, w.out, Y};
  const dim3 grid(static_cast<unsigned>(w.out / 64), static_cast<unsigned>((M + kMvTok - 1) / kMvTok));
  timing_before(QLORA_KERNEL_MATVEC, stream);
  matvec_kernel<<<grid, kMvThreads, 0, stream>>>(a);
  timing_after(QLORA_KERNEL_MATVEC, stream);
  count_launch();
  return cudaGetLastError();
}

}  // namespace qlora
