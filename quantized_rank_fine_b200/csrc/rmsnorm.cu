// Residual addition with RMS norm, forward and gradient: what stands between two
// adapted linears.
//
//   h = bf16(res + keep x / (1 - p)),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd g
//   out: h (bf16), bf16(y), and y in 8 bits: per row or per 64 columns
//        s = fl32(max|y| / 448), code = E4M3(fl32(y / s))
//   gh = g dy,  c = mean(gh h) rstd^2,  dh = rstd (gh - h c) + dH
//   out: dR = bf16(dh), dX = bf16(keep dh / (1 - p)), dG = sum over rows of dy h rstd
//
// Both are bound by streaming the rows once (a few flops and bytes an element).
// A CTA takes a row: every thread holds its 16-byte vectors of the row in
// registers, so the row is read once however many passes the arithmetic takes.
#include "common.cuh"
#include "kernels.h"
#include "philox.cuh"

namespace qlora {

namespace {

constexpr int kNormMaxThreads = 1024;

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// The gain of columns 8v .. 8v+7.
__device__ __forceinline__ void load_gain(const void* G, bool f32, int v, float (&g)[8]) {
  if (f32) {
    const float4 a = reinterpret_cast<const float4*>(G)[2 * v], b = reinterpret_cast<const float4*>(G)[2 * v + 1];
    g[0] = a.x;
    g[1] = a.y;
    g[2] = a.z;
    g[3] = a.w;
    g[4] = b.x;
    g[5] = b.y;
    g[6] = b.z;
    g[7] = b.w;
  } else {
    unpack8(reinterpret_cast<const uint4*>(G)[v], g);
  }
}

// keep * scale of the eight elements from e (a multiple of 8).
__device__ __forceinline__ void keep8(const DropoutCounter& d, uint64_t off, float scale, int64_t e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = philox4x32_10(static_cast<uint64_t>(e / 4 + i), off, d.seed);
    f[4 * i] = u.x >= d.threshold ? scale : 0.0f;
    f[4 * i + 1] = u.y >= d.threshold ? scale : 0.0f;
    f[4 * i + 2] = u.z >= d.threshold ? scale : 0.0f;
    f[4 * i + 3] = u.w >= d.threshold ? scale : 0.0f;
  }
}

// res + x k, ready to be rounded to bf16.  A binary32 sum that is a tie between two
// bf16 values may stand for an exact sum on either side of it, and under dropout
// many do (x / (1 - p) often lies within 2^-26 of a short number): such a sum is
// formed again in 64 bits and moved off the tie, so that the stored h is the
// nearest bf16 to the exact sum.  A sum that is not a tie cannot be on the wrong
// side of one, as ties are binary32 numbers and rounding is monotone.
__device__ __forceinline__ float add_kept(float res, float x, float k) {
  float s = fmaf(x, k, res);
  if ((__float_as_uint(s) & 0xFFFFu) == 0x8000u) {
    const double t = static_cast<double>(x) * static_cast<double>(k) + static_cast<double>(res);
    const double sd = static_cast<double>(s);
    if (t != sd) s = __uint_as_float(__float_as_uint(s) + (((t > sd) == (s > 0.0f)) ? 1u : 0xFFFFFFFFu));
  }
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA (every thread gets it); `red` has 32 floats.  The first barrier
// lets `red` be used again.
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  v = warp_sum(v);
  if (nw == 1) return v;
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < nw ? red[lane] : 0.0f);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  v = __reduce_max_sync(0xffffffffu, v);
  if (nw == 1) return v;
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

// Largest |y| of eight values as bits: unsigned order is the order of magnitudes,
// with infinity and NaN above every number, so a block that holds one gets an
// infinite or NaN scale and dequantises to NaN instead of hiding it.
__device__ __forceinline__ uint32_t max_bits8(const float (&y)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  return a;
}

__device__ __forceinline__ uint2 e4m3_codes(const float (&y)[8], float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 q = make_float2(0.0f, 0.0f);
    if (s != 0.0f) q = make_float2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
    w[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// VPT vectors of 8 columns a thread; kQuant: 0 none, 1 one scale a row, 2 one per 64 columns.
template <int VPT, bool kDrop, int kQuant>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_fwd_kernel(const NormFwd p) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const int nv = static_cast<int>(p.n / 8);
  const uint4* X = reinterpret_cast<const uint4*>(p.X + row * p.n);
  const uint4* R = p.R ? reinterpret_cast<const uint4*>(p.R + row * p.n) : nullptr;
  const uint64_t off = kDrop ? dropout_offset(p.drop) : 0;
  uint4 h[VPT];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    h[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < nv) {
      h[i] = X[v];
      float x[8], f[8];
      unpack8(h[i], x);
      if (kDrop || R) {
        float res[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (R) unpack8(R[v], res);
        if (kDrop) {
          float k[8];
          keep8(p.drop, off, p.keep_scale, row * p.n + 8 * v, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = add_kept(res[j], x[j], k[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = res[j] + x[j];
        }
        h[i] = pack8(f);
        if (p.H) reinterpret_cast<uint4*>(p.H + row * p.n)[v] = h[i];
        unpack8(h[i], x);
      } else if (p.H) {
        reinterpret_cast<uint4*>(p.H + row * p.n)[v] = h[i];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    }
  }
  const float mean = __fdiv_rn(block_sum(ss, red), static_cast<float>(p.n));
  const float rstd = __frsqrt_rn(mean + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;

  uint32_t top = 0;
  if (kQuant == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nv) {
        float x[8], g[8];
        unpack8(h[i], x);
        load_gain(p.G, p.g_f32, v, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * rstd * g[j];
        top = max(top, max_bits8(x));
      }
    }
    top = block_max(top, reinterpret_cast<uint32_t*>(red));
    if (threadIdx.x == 0) p.q_scales[row] = __fdiv_rn(__uint_as_float(top), 448.0f);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (v < nv) {
      float g[8];
      unpack8(h[i], y);
      load_gain(p.G, p.g_f32, v, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = y[j] * rstd * g[j];
      if (p.Y) reinterpret_cast<uint4*>(p.Y + row * p.n)[v] = pack8(y);
    }
    if (kQuant == 2) {
      // a block of 64 columns is 8 neighbouring lanes (n is a multiple of 64)
      top = max_bits8(y);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (kQuant && v < nv) {
      const float s = __fdiv_rn(__uint_as_float(top), 448.0f);
      reinterpret_cast<uint2*>(p.Q + row * p.n)[v] = e4m3_codes(y, s);
      if (kQuant == 2 && (v & 7) == 0) p.q_scales[row * (p.n / 64) + v / 8] = s;
    }
  }
}

// One CTA walks the rows blockIdx.x, + gridDim.x, ...; the gain's gradient of a
// thread's columns stays in registers over them and goes to the CTA's row of `parts`.
template <int VPT, bool kDrop>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_bwd_kernel(const NormBwd p) {
  __shared__ float red[32];
  const int nv = static_cast<int>(p.n / 8);
  const uint64_t off = kDrop ? dropout_offset(p.drop) : 0;
  float dg[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float rstd = p.rstd[row];
    uint4 h[VPT], dy[VPT];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nv) {
        h[i] = reinterpret_cast<const uint4*>(p.H + row * p.n)[v];
        dy[i] = reinterpret_cast<const uint4*>(p.dY + row * p.n)[v];
        float x[8], d[8], g[8];
        unpack8(h[i], x);
        unpack8(dy[i], d);
        load_gain(p.G, p.g_f32, v, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          c = fmaf(d[j] * g[j], x[j], c);
          dg[i][j] = fmaf(d[j], x[j] * rstd, dg[i][j]);
        }
      }
    }
    c = __fdiv_rn(block_sum(c, red), static_cast<float>(p.n)) * rstd * rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nv) {
        float x[8], d[8], g[8];
        unpack8(h[i], x);
        unpack8(dy[i], d);
        load_gain(p.G, p.g_f32, v, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = rstd * fmaf(-c, x[j], d[j] * g[j]);
        if (p.dH) {
          float e[8];
          unpack8(reinterpret_cast<const uint4*>(p.dH + row * p.n)[v], e);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += e[j];
        }
        reinterpret_cast<uint4*>(p.dR + row * p.n)[v] = pack8(d);
        if (kDrop && p.dX) {
          float k[8];
          keep8(p.drop, off, p.keep_scale, row * p.n + 8 * v, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] *= k[j];
          reinterpret_cast<uint4*>(p.dX + row * p.n)[v] = pack8(d);
        }
      }
    }
  }
  if (p.dG) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nv) {
        float4* o = reinterpret_cast<float4*>(p.parts + static_cast<int64_t>(blockIdx.x) * p.n) + 2 * v;
        o[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
        o[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
      }
    }
  }
}

// dG[col] = the sum of the parts in CTA order (the same bits every time).
__global__ void __launch_bounds__(256) rmsnorm_dgain_kernel(const float* parts, int nparts, int64_t n, float* dG,
                                                            int accumulate) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (col >= n) return;
  float s = 0.0f;
  for (int i = 0; i < nparts; ++i) s += parts[i * n + col];
  dG[col] = accumulate ? dG[col] + s : s;
}

constexpr int kNormParts = 296;   // most CTAs of the gradient (two per SM)

// Vectors a thread holds and the threads of a CTA for rows of nv vectors.
void norm_plan(int64_t nv, int& vpt, int& threads) {
  vpt = nv <= 1024 ? 1 : (nv <= 2048 ? 2 : (nv <= 4096 ? 4 : 8));
  threads = static_cast<int>(((nv + vpt - 1) / vpt + 31) / 32 * 32);
}

template <int VPT>
void run_fwd(const NormFwd& a, int threads, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.M));
  const int quant = a.Q ? (a.q_block ? 2 : 1) : 0;
  if (a.drop.on) {
    if (quant == 0) rmsnorm_fwd_kernel<VPT, true, 0><<<grid, threads, 0, stream>>>(a);
    else if (quant == 1) rmsnorm_fwd_kernel<VPT, true, 1><<<grid, threads, 0, stream>>>(a);
    else rmsnorm_fwd_kernel<VPT, true, 2><<<grid, threads, 0, stream>>>(a);
  } else {
    if (quant == 0) rmsnorm_fwd_kernel<VPT, false, 0><<<grid, threads, 0, stream>>>(a);
    else if (quant == 1) rmsnorm_fwd_kernel<VPT, false, 1><<<grid, threads, 0, stream>>>(a);
    else rmsnorm_fwd_kernel<VPT, false, 2><<<grid, threads, 0, stream>>>(a);
  }
}

template <int VPT>
void run_bwd(const NormBwd& a, int grid, int threads, cudaStream_t stream) {
  if (a.drop.on) rmsnorm_bwd_kernel<VPT, true><<<grid, threads, 0, stream>>>(a);
  else rmsnorm_bwd_kernel<VPT, false><<<grid, threads, 0, stream>>>(a);
}

int bwd_grid(int64_t M) { return static_cast<int>(std::min<int64_t>(M, kNormParts)); }

}  // namespace

size_t norm_bwd_parts_bytes(int64_t M, int64_t n) { return static_cast<size_t>(bwd_grid(M)) * n * sizeof(float); }

cudaError_t launch_rmsnorm_fwd(const NormFwd& a, cudaStream_t stream) {
  int vpt, threads;
  norm_plan(a.n / 8, vpt, threads);
  timing_before(QLORA_KERNEL_RMSNORM, stream);
  if (vpt == 1) run_fwd<1>(a, threads, stream);
  else if (vpt == 2) run_fwd<2>(a, threads, stream);
  else if (vpt == 4) run_fwd<4>(a, threads, stream);
  else run_fwd<8>(a, threads, stream);
  timing_after(QLORA_KERNEL_RMSNORM, stream);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_bwd(const NormBwd& a, cudaStream_t stream) {
  int vpt, threads;
  norm_plan(a.n / 8, vpt, threads);
  const int grid = bwd_grid(a.M);
  timing_before(QLORA_KERNEL_RMSNORM_BWD, stream);
  if (vpt == 1) run_bwd<1>(a, grid, threads, stream);
  else if (vpt == 2) run_bwd<2>(a, grid, threads, stream);
  else if (vpt == 4) run_bwd<4>(a, grid, threads, stream);
  else run_bwd<8>(a, grid, threads, stream);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.dG) {
    rmsnorm_dgain_kernel<<<static_cast<unsigned>((a.n + 255) / 256), 256, 0, stream>>>(a.parts, grid, a.n, a.dG,
                                                                                      a.accumulate ? 1 : 0);
    count_launch();
    e = cudaGetLastError();
  }
  timing_after(QLORA_KERNEL_RMSNORM_BWD, stream);
  return e;
}

}  // namespace qlora
