// Residual addition with RMS norm, forward and gradient: what stands between two
// adapted linears.
//
//   h = bf16(res + keep x / (1 - p)),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd g
//   out: h (bf16), bf16(y), and y in 8 bits: per row or per 64 columns
//        s = fl32(max|y| / 448), code = E4M3(fl32(y / s))
//   gh = g dy,  c = mean(gh h) rstd^2,  dh = rstd (gh - h c) + dH
//   out: dR = bf16(dh), dX = bf16(keep dh / (1 - p)), dG = sum over rows of dy h rstd
//
// The floor of both is to stream the rows once (a few flops and bytes an element).
// A CTA takes a row: every thread holds its 16-byte vectors of the row in
// registers, so the row is read once however many passes the arithmetic takes.
// The gradient's CTAs walk several rows with the next row's loads in flight, and
// keep their columns of the gain and of its gradient in registers; the parts of
// the CTAs are added by a second, programmatically dependent launch.
//
// Measured (graph of calls over rows larger than L2): forward 2048 x 4096 12.8 us (5.2
// TB/s of 8 bytes an element); gradient 8192 x 4096 43.6 us (6.2 TB/s) and 4.7 more
// with the gain's.  Dropout adds Philox's ten rounds for four elements: forward
// 8192 x 4096 51 us, with bf16 and 8-bit output 66, gradient 69 with the gain's; then 71
// and 62% of the cycles issue an instruction and DRAM runs at 51 and 55% of its peak.
// Not at the floor either: short rows forward, where every row has a CTA of its own
// (8192 x 512 9.2 us of 5.1, 65536 x 64 68 of 5; the gradient without the gain's,
// several rows a CTA, 6.9 and 19); rows past 8192 columns, where one CTA of up to 1024
// threads fits on an SM and nothing covers a row's latency but the next row (2048 x
// 16384 forward 51 us of 41, gradient 71; 512 x 65536 58 and 134); and the gain's
// gradient, whose parts pass through memory once more (2048 x 4096 15.9 us, 11.6 without).
#include "common.cuh"
#include "kernels.h"
#include "philox.cuh"
#include "sm100.cuh"

namespace qlora {

namespace {

using namespace sm100;

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

// Two fp32 operations as one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%6, %7};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
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

// The random words of the eight elements from e (a multiple of 8).
__device__ __forceinline__ void words8(const DropoutCounter& d, uint64_t off, int64_t e, uint32_t (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = philox4x32_10(static_cast<uint64_t>(e / 4 + i), off, d);
    u[4 * i] = w.x;
    u[4 * i + 1] = w.y;
    u[4 * i + 2] = w.z;
    u[4 * i + 3] = w.w;
  }
}

// res + x scale of eight kept elements (res of the dropped ones, whatever x holds),
// ready to be rounded to bf16: the sum is rounded to odd in binary32 (of its two
// neighbours the one with an odd last bit, where it is not exact), so that the second
// rounding sees on which side of a tie between two bf16 values it lies.  Under dropout
// many sums lie next to one: x / (1 - p) is often within 2^-26 of a short number.
__device__ __forceinline__ void add_kept8(const float (&res)[8], const float (&x)[8], const uint32_t (&u)[8],
                                          uint32_t threshold, float scale, float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float lo = __fmaf_rd(x[j], scale, res[j]), hi = __fmaf_ru(x[j], scale, res[j]);
    const float odd = (__float_as_uint(lo) & 1u) ? lo : hi;
    s[j] = u[j] >= threshold ? odd : res[j];
  }
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

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The scale of a block whose largest |y| has these bits, zero below the normal numbers.
__device__ __forceinline__ float block_scale(uint32_t top) {
  const float s = __fdiv_rn(__uint_as_float(top), 448.0f);
  return s < 0x1p-126f ? 0.0f : s;
}

// E4M3(fl32(y / s)) of eight values, 0 where s = 0.  The quotients by Markstein's
// theorem (IBM Journal of Research and Development 34, 1990): with the reciprocal r
// of s, the product q = y r and the rest y - q s, each rounded once, q + (y - q s) r
// is the correctly rounded quotient, as long as the rest does not underflow (|y|
// above about 2^-100).  A block of tiny values is therefore brought up by a power of
// two, y and s alike; above, a y whose rest underflows is far below the smallest code.
__device__ __forceinline__ uint2 e4m3_codes(const float (&v)[8], float s) {
  if (s == 0.0f) return make_uint2(0u, 0u);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i];
  if (s < 0x1p-60f) {
    s *= 0x1p64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= 0x1p64f;
  }
  const float inv = __frcp_rn(s);
  const float2 r2 = make_float2(inv, inv), s2 = make_float2(-s, -s);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = make_float2(y[2 * i], y[2 * i + 1]), q0 = mul2(u, r2);
    const float2 q = fma2(fma2(q0, s2, u), r2, q0);
    w[i] = e4m3_pair(q.x, q.y);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// bf16(a + b) of pairs, one rounding.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A thread's vectors of the row between the passes: as fp32 where they are few (they
// are unpacked once), as bf16 pairs where they are many.
template <int VPT, bool kWide>
struct Held;
template <int VPT>
struct Held<VPT, true> {
  float f[VPT][8];
  __device__ __forceinline__ void set(int i, uint4, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = v[j];
  }
  __device__ __forceinline__ void get(int i, float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[i][j];
  }
};
template <int VPT>
struct Held<VPT, false> {
  uint4 p[VPT];
  __device__ __forceinline__ void set(int i, uint4 v, const float (&)[8]) { p[i] = v; }
  __device__ __forceinline__ void get(int i, float (&v)[8]) const { unpack8(p[i], v); }
};

// VPT vectors of 8 columns a thread; kQuant: 0 none, 1 one scale a row, 2 one per 64 columns.
template <int VPT, bool kDrop, int kQuant>
__global__ void __launch_bounds__(VPT == 2 ? 512 : kNormMaxThreads) rmsnorm_fwd_kernel(const __grid_constant__ NormFwd p) {
  __shared__ float red[32];
  grid_launch_dependents();   // they wait for this kernel to finish, as it waits for the one before
  grid_dependency_wait();
  const int64_t row = blockIdx.x;
  const int nv = static_cast<int>(p.n / 8);
  const uint4* X = reinterpret_cast<const uint4*>(p.X + row * p.n);
  const uint4* R = p.R ? reinterpret_cast<const uint4*>(p.R + row * p.n) : nullptr;
  const uint64_t off = kDrop ? dropout_offset(p.drop) : 0;
  Held<VPT, (VPT <= 2)> held;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    uint4 h = make_uint4(0u, 0u, 0u, 0u);
    if (v < nv) {
      h = X[v];
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (R) r = R[v];
      if constexpr (kDrop) {
        float res[8], s[8];
        uint32_t u[8];
        unpack8(h, x);
        unpack8(r, res);
        words8(p.drop, off, row * p.n + 8 * v, u);
        add_kept8(res, x, u, p.drop.threshold, p.keep_scale, s);
        h = pack8(s);
      } else if (R) {
        h = make_uint4(add_bf16x2(h.x, r.x), add_bf16x2(h.y, r.y), add_bf16x2(h.z, r.z), add_bf16x2(h.w, r.w));
      }
      if (p.H) reinterpret_cast<uint4*>(p.H + row * p.n)[v] = h;
      unpack8(h, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    }
    held.set(i, h, x);
  }
  const float mean = __fdiv_rn(block_sum(ss, red), static_cast<float>(p.n));
  const float rstd = __frsqrt_rn(mean + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;

  // y of a vector, (h rstd) g
  auto normed = [&](int i, int v, float (&y)[8]) {
    float h[8], g[8];
    held.get(i, h);
    load_gain(p.G, p.g_f32, v, g);
    const float2 rr = make_float2(rstd, rstd);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 o = mul2(mul2(make_float2(h[j], h[j + 1]), rr), make_float2(g[j], g[j + 1]));
      y[j] = o.x;
      y[j + 1] = o.y;
    }
  };
  uint32_t top = 0;
  if constexpr (kQuant == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nv) {
        float y[8];
        normed(i, v, y);
        if constexpr (VPT <= 2) held.set(i, make_uint4(0u, 0u, 0u, 0u), y);   // y takes the place of h
        top = max(top, max_bits8(y));
      }
    }
    top = block_max(top, reinterpret_cast<uint32_t*>(red));
    if (threadIdx.x == 0) p.q_scales[row] = block_scale(top);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (v < nv) {
      if constexpr (kQuant == 1 && VPT <= 2) held.get(i, y);
      else normed(i, v, y);
      if (p.Y) reinterpret_cast<uint4*>(p.Y + row * p.n)[v] = pack8(y);
    }
    if constexpr (kQuant == 2) {
      // a block of 64 columns is 8 neighbouring lanes (n is a multiple of 64)
      top = max_bits8(y);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (kQuant && v < nv) {
      const float s = block_scale(top);
      reinterpret_cast<uint2*>(p.Q + row * p.n)[v] = e4m3_codes(y, s);
      if (kQuant == 2 && (v & 7) == 0) p.q_scales[row * (p.n / 64) + v / 8] = s;
    }
  }
}

constexpr int kBwdThreads = 512;    // of a CTA that takes several short rows at once
constexpr int kBwdMaxCluster = 8;   // CTAs that share a row of more than 8192 columns

struct BwdPlan {
  int threads;    // a row's threads in a CTA, one vector of 8 columns each
  int groups;     // rows a CTA takes at once
  int cluster;    // CTAs that share a row
  int ctas;       // CTAs (or clusters), each with its row of `parts`
};

// Threads for one vector each: a short row leaves room for several in a CTA of 512
// threads (two CTAs an SM), a row of up to 8192 columns has a CTA to itself, and a
// longer one is split over a cluster (one CTA an SM).
BwdPlan bwd_plan(int64_t M, int64_t n) {
  const int nv = static_cast<int>(n / 8);
  BwdPlan b{};
  b.cluster = nv <= 1024 ? 1 : (nv <= 2048 ? 2 : (nv <= 4096 ? 4 : 8));
  b.threads = ((nv + b.cluster - 1) / b.cluster + 31) / 32 * 32;
  b.groups = b.threads <= kBwdThreads / 2 ? kBwdThreads / b.threads : 1;
  const int64_t most = b.threads <= kBwdThreads ? 296 : 148 / b.cluster;
  b.ctas = static_cast<int>(std::min<int64_t>((M + b.groups - 1) / b.groups, most));
  return b;
}

// A group of `threads` threads walks the rows blockIdx.x groups + its number, ... (a
// cluster of kCluster CTAs the rows of its own number), one vector a thread, with the
// next row's loads in flight; the gain's gradient of a thread's columns stays in
// registers and goes to the CTA's row of `parts`.
template <bool kDrop, bool kCluster>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_bwd_kernel(const __grid_constant__ NormBwd p,
                                                                      const int threads, const int groups) {
  __shared__ float red[2][kCluster ? 32 * kBwdMaxCluster : 32];
  __shared__ float4 sums[kCluster ? 1 : kBwdThreads * 2];
  if constexpr (kCluster) cluster_started_arrive();
  grid_launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = threads >> 5;
  const int group = kCluster ? 0 : threadIdx.x / threads;
  const int C = kCluster ? static_cast<int>(cluster_nctarank()) : 1, rank = kCluster ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t step = kCluster ? gridDim.x / C : static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = kCluster ? blockIdx.x / C : static_cast<int64_t>(blockIdx.x) * groups;
  const int v = rank * threads + threadIdx.x - group * threads;   // vector of the row
  const bool mine = v < static_cast<int>(p.n / 8);
  const uint64_t off = kDrop ? dropout_offset(p.drop) : 0;
  const float cols = static_cast<float>(p.n);
  float dg[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, g[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  uint4 h, dy, dh;
  float rstd;
  auto load = [&](int64_t row) {
    h = dy = dh = make_uint4(0u, 0u, 0u, 0u);
    rstd = 0.0f;
    if (row < p.M) {
      rstd = p.rstd[row];
      if (mine) {
        h = reinterpret_cast<const uint4*>(p.H + row * p.n)[v];
        dy = reinterpret_cast<const uint4*>(p.dY + row * p.n)[v];
        if (p.dH) dh = reinterpret_cast<const uint4*>(p.dH + row * p.n)[v];
      }
    }
  };
  if (mine) load_gain(p.G, p.g_f32, v, g);
  int flip = 0;
  load(first + group);
  if constexpr (kCluster) cluster_started_wait();
  for (int64_t r0 = first; r0 < p.M; r0 += step, flip ^= 1) {   // the same turns for every thread
    const int64_t row = r0 + group;
    const float rs = rstd;
    const uint4 x4 = h, d4 = dy, e4 = dh;
    float x[8], d[8];
    unpack8(x4, x);
    unpack8(d4, d);
    float2 c2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 xj = make_float2(x[j], x[j + 1]), dj = make_float2(d[j], d[j + 1]);
      c2 = fma2(mul2(dj, make_float2(g[j], g[j + 1])), xj, c2);
      const float2 s = fma2(dj, mul2(xj, make_float2(rs, rs)), make_float2(dg[j], dg[j + 1]));
      dg[j] = s.x;
      dg[j + 1] = s.y;
    }
    load(row + step);
    // A cluster's barrier is a long wait with one CTA an SM: the row's mask is formed
    // before it (2048 x 16384: 108 -> 90 us).  Other CTAs fill an SM's wait at a
    // CTA's barrier, where packing the mask into bits only costs (8192 x 4096: 69 -> 79).
    uint32_t kept = 0;
    if (kCluster && kDrop && p.dX && row < p.M) {
      uint32_t u[8];
      words8(p.drop, off, row * p.n + 8 * v, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) kept |= u[j] >= p.drop.threshold ? 1u << j : 0u;
    }
    // two sets of warp sums in turn: a row's are not written before every thread has
    // read those of the row before the last
    float c = warp_sum(c2.x + c2.y);
    if constexpr (kCluster) {
      if (lane < C) st_shared_cluster_f32(mapa_shared(smem_addr(&red[flip][rank * 32 + warp]), lane), c);
      cluster_sync();
      c = 0.0f;
      for (int i = 0; i < C; ++i) c += lane < nw ? red[flip][i * 32 + lane] : 0.0f;
      c = warp_sum(c);
    } else {
      if (lane == 0) red[flip][warp] = c;
      __syncthreads();
      c = warp_sum(lane < nw ? red[flip][group * nw + lane] : 0.0f);
    }
    c = __fdiv_rn(c, cols) * rs * rs;
    if (mine && row < p.M) {
      float e[8];
      unpack8(x4, x);
      unpack8(d4, d);
      unpack8(e4, e);   // zeros without dH
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 gd = mul2(make_float2(d[j], d[j + 1]), make_float2(g[j], g[j + 1]));
        const float2 o = fma2(make_float2(rs, rs), fma2(make_float2(-c, -c), make_float2(x[j], x[j + 1]), gd),
                              make_float2(e[j], e[j + 1]));
        d[j] = o.x;
        d[j + 1] = o.y;
      }
      reinterpret_cast<uint4*>(p.dR + row * p.n)[v] = pack8(d);
      if (kDrop && p.dX) {
        uint32_t u[8];
        if constexpr (!kCluster) words8(p.drop, off, row * p.n + 8 * v, u);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          d[j] = (kCluster ? (kept >> j) & 1u : u[j] >= p.drop.threshold) ? d[j] * p.keep_scale : 0.0f;
        reinterpret_cast<uint4*>(p.dX + row * p.n)[v] = pack8(d);
      }
    }
  }
  if (!p.dG) return;
  if (!kCluster && groups > 1) {
    // the groups of this CTA, added in order by the first
    sums[2 * threadIdx.x] = make_float4(dg[0], dg[1], dg[2], dg[3]);
    sums[2 * threadIdx.x + 1] = make_float4(dg[4], dg[5], dg[6], dg[7]);
    __syncthreads();
    if (group > 0) return;
    for (int i = 1; i < groups; ++i) {
      const float4 a = sums[2 * (threadIdx.x + i * threads)], b = sums[2 * (threadIdx.x + i * threads) + 1];
      dg[0] += a.x;
      dg[1] += a.y;
      dg[2] += a.z;
      dg[3] += a.w;
      dg[4] += b.x;
      dg[5] += b.y;
      dg[6] += b.z;
      dg[7] += b.w;
    }
  }
  if (mine) {
    float4* o = reinterpret_cast<float4*>(p.parts + static_cast<int64_t>(blockIdx.x / C) * p.n) + 2 * v;
    o[0] = make_float4(dg[0], dg[1], dg[2], dg[3]);
    o[1] = make_float4(dg[4], dg[5], dg[6], dg[7]);
  }
}

// dG[col] = the sum of the parts.  A CTA takes 16 columns (4 threads of 4) with 64 row
// lanes: lane l adds the parts l, l + 64, ...; the lanes of a warp and then the warps
// are added in a fixed order, so the bits are the same every time.
__global__ void __launch_bounds__(256) rmsnorm_dgain_kernel(const float4* parts, int nparts, int64_t n, float4* dG,
                                                            int accumulate) {
  __shared__ float4 red[8][4];
  grid_launch_dependents();
  grid_dependency_wait();
  const int c = threadIdx.x & 3, l = threadIdx.x >> 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t nq = n / 4, q = static_cast<int64_t>(blockIdx.x) * 4 + c;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (q < nq) {
#pragma unroll 5
    for (int i = l; i < nparts; i += 64) {
      const float4 v = __ldcg(parts + i * nq + q);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
  }
  if (lane < 4) red[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x >= 4 || q >= nq) return;
  s = red[0][c];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const float4 v = red[i][c];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  if (accumulate) {
    const float4 v = dG[q];
    s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
  }
  dG[q] = s;
}

// Launch as a programmatic dependent (the kernels wait before they touch memory), in
// clusters of `cluster` CTAs.
template <typename... P, typename... A>
void launch_dependent(void (*kernel)(P...), unsigned grid, unsigned threads, unsigned cluster, cudaStream_t stream,
                      A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kernel, args...);   // a failure is the last error, read by the caller
}

// Vectors a thread holds and the threads of a CTA for rows of nv vectors.  Forward:
// one vector a thread while there are fewer rows than would fill the SMs (a row's
// latency counts: 1 x 4096, 2.6 us against 3.4 with two), else two (2048 x 4096, 10.8
// us against 12.9: twice the CTAs lie on an SM); more only where a row has more than a
// CTA's threads hold.
void fwd_plan(int64_t M, int64_t nv, int& vpt, int& threads) {
  vpt = M < 592 && nv <= 1024 ? 1 : (nv <= 1024 ? 2 : (nv <= 4096 ? 4 : 8));
  threads = static_cast<int>(((nv + vpt - 1) / vpt + 31) / 32 * 32);
}

template <int VPT>
void run_fwd(const NormFwd& a, int threads, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.M);
  const int quant = a.Q ? (a.q_block ? 2 : 1) : 0;
  if (a.drop.on) {
    if (quant == 0) launch_dependent(rmsnorm_fwd_kernel<VPT, true, 0>, grid, threads, 1, stream, a);
    else if (quant == 1) launch_dependent(rmsnorm_fwd_kernel<VPT, true, 1>, grid, threads, 1, stream, a);
    else launch_dependent(rmsnorm_fwd_kernel<VPT, true, 2>, grid, threads, 1, stream, a);
  } else {
    if (quant == 0) launch_dependent(rmsnorm_fwd_kernel<VPT, false, 0>, grid, threads, 1, stream, a);
    else if (quant == 1) launch_dependent(rmsnorm_fwd_kernel<VPT, false, 1>, grid, threads, 1, stream, a);
    else launch_dependent(rmsnorm_fwd_kernel<VPT, false, 2>, grid, threads, 1, stream, a);
  }
}

}  // namespace

size_t norm_bwd_parts_bytes(int64_t M, int64_t n) { return static_cast<size_t>(bwd_plan(M, n).ctas) * n * sizeof(float); }

cudaError_t launch_rmsnorm_fwd(const NormFwd& a, cudaStream_t stream) {
  int vpt, threads;
  fwd_plan(a.M, a.n / 8, vpt, threads);
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
  const BwdPlan b = bwd_plan(a.M, a.n);
  const unsigned grid = static_cast<unsigned>(b.ctas * b.cluster), threads = static_cast<unsigned>(b.threads * b.groups);
  timing_before(QLORA_KERNEL_RMSNORM_BWD, stream);
  if (b.cluster > 1)
    launch_dependent(a.drop.on ? rmsnorm_bwd_kernel<true, true> : rmsnorm_bwd_kernel<false, true>, grid, threads,
                     static_cast<unsigned>(b.cluster), stream, a, b.threads, b.groups);
  else
    launch_dependent(a.drop.on ? rmsnorm_bwd_kernel<true, false> : rmsnorm_bwd_kernel<false, false>, grid, threads, 1,
                     stream, a, b.threads, b.groups);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.dG) {
    launch_dependent(rmsnorm_dgain_kernel, static_cast<unsigned>((a.n + 15) / 16), 256, 1, stream,
                     reinterpret_cast<const float4*>(a.parts), b.ctas, a.n, reinterpret_cast<float4*>(a.dG),
                     a.accumulate ? 1 : 0);
    count_launch();
    e = cudaGetLastError();
  }
  timing_after(QLORA_KERNEL_RMSNORM_BWD, stream);
  return e;
}

}  // namespace qlora
