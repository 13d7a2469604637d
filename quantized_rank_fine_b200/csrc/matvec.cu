// A few tokens (M <= 16) through a weight of 4-bit integers with one scale per 16:
//
//   Y[m][n] = sum_k x[m][k] q[k][n] s[k][n / 16] + sum_j V[m][j] B[j][n],  V = scale X A
//
// bound by reading the codes and scales once (0.75 B a weight).
//
//   * Split over K without a second pass: both terms are linear in the rows, so a
//     CTA that owns the rows [k0, k0 + Kc) of a 256-column tile forms x W of its
//     rows and also V of its rows times B; the parts of a tile are added over a
//     thread-block cluster in split order.  One launch, no scratch, no atomics.
//   * Every warp is its own stream: warp (ks, half) takes the 16-row steps ks,
//     ks + 4, ... of its CTA's rows and 128 of the 256 columns, and copies just
//     those codes, scales, x and A into its own ring with cp.async.  Nothing but
//     __syncwarp orders a stage, so there is no barrier to wait on in the loop.
//   * Tensor cores with the weight as the 16 x 16 A operand and 8 tokens as the B
//     operand: mma.sync m16n8k16 (128-row tcgen05 tiles have no use for 16 tokens).
//     The 16 operand rows are the 16 columns that share a scale, so the scale
//     folds into x: B = bf16(x s), and A is the integer q itself, exact in bf16.
//     The byte transpose of ldmatrix (m16n16 .b8) hands lane (g, t) one byte, two
//     columns, of rows 4t .. 4t+3; a byte permute sets the nibble into bf16 128 + code
//     and one packed subtraction of 136 leaves q.
//   * x s is rounded to bf16 (2^-9 of each product at most, signs independent), the
//     same size as the output's own rounding; sums are fp32.  x itself and V are not
//     rounded in a way that reaches Y: V goes in as a sum of two bf16 numbers.
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

#include <mutex>

namespace qlora {

namespace {

using namespace sm100;

constexpr int kMvWarps = 8;                     // 4 row steps x 2 column halves
constexpr int kMvThreads = kMvWarps * 32;
constexpr int kMvTile = 256;                    // columns per CTA
constexpr int kMvRows = 64;                     // rows per stage of a CTA (16 per warp)
constexpr int kMvMaxCluster = 16;
constexpr uint32_t kMvCodePitch = 80;           // 64 bytes of codes a row; 80 keeps 8 rows on different banks

struct MvArgs {
  const uint8_t* codes;
  const float* scales;
  const void* x;
  const float* x_scales;
  int x_block;
  const uint16_t* A;
  const uint16_t* B;
  int M, r;
  float scale;
  int64_t K, N;
  int64_t Kc;             // rows per split (multiple of 64)
  uint16_t* Y;
  uint16_t* V;            // saved V, or nullptr
};

// MT: token tiles of 8.  RCH: adapter columns per column half (0: no adapter).
// X8: x in E4M3 codes with scales, else bf16.
template <int MT, int RCH, bool X8>
struct MvLayout {
  static constexpr uint32_t kScale = 16 * kMvCodePitch;            // 16 rows x 8 scales
  static constexpr uint32_t kX = kScale + 512;                     // tokens x 16 k
  static constexpr uint32_t kXPitch = X8 ? 16 : 32;
  static constexpr uint32_t kA = kX + MT * 8 * kXPitch;            // 16 rows x RCH, padded
  static constexpr uint32_t kAPitch = RCH * 2 + 16;
  static constexpr uint32_t kSlot = kA + (RCH ? 16 * kAPitch : 0);
  static constexpr uint32_t kVs = 4 * 2 * RCH * MT * 8 * 4;        // V of the 4 row steps
  static constexpr uint32_t kTail = kVs + 4 * MT * 8 * kMvTile * 4;   // and the 4 partial tiles
  static constexpr uint32_t kRecv = (MT * 8 * 64 + MT * 8 * 2 * RCH / 4 + kMvMaxCluster) * 16;
  static constexpr uint32_t bytes(int depth) {
    return (kMvWarps * depth * kSlot > kTail ? kMvWarps * depth * kSlot : kTail) + kRecv;
  }
  static constexpr int depth(uint32_t budget) {
    int d = 6;
    while (d > 2 && bytes(d) > budget) --d;
    return d;
  }
  // ring depth for two CTAs on an SM, or for one where that leaves too few stages
  static constexpr int kTwo = depth(113 * 1024);
  static constexpr int kDepth = kTwo >= 3 ? kTwo : depth(226 * 1024);
  static constexpr uint32_t kSmem = bytes(kDepth);
  static constexpr int kCtas = kTwo >= 3 ? 2 : 1;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// (a.x b, a.y b) as one packed multiplication
__device__ __forceinline__ float2 mul2(float2 a, float b) {
  float2 d;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b));
  return d;
}

__device__ __forceinline__ float4 lds128(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// bf16(v) and bf16(v - bf16(v)) of two values, packed: together 16 bits of each.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(v0, v1);
  lo = pack_bf16x2(v0 - bf16_lo(hi), v1 - bf16_hi(hi));
}

template <int MT, int RCH, bool X8>
__global__ void __launch_bounds__(kMvThreads, MvLayout<MT, RCH, X8>::kCtas) matvec_kernel(const MvArgs p) {
  using L = MvLayout<MT, RCH, X8>;
  constexpr int D = L::kDepth;
  constexpr int RT = RCH / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* recv = smem + (L::kSmem - L::kRecv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int ks = warp & 3, half = warp >> 2;
  const int tile = blockIdx.x, split = blockIdx.y;
  const int64_t kbeg = split * p.Kc;
  const int nst = static_cast<int>((p.K - kbeg < p.Kc ? p.K - kbeg : p.Kc) / kMvRows);
  const int64_t col0 = static_cast<int64_t>(tile) * kMvTile + half * 128;   // first column of this warp

  // The kernels after this one wait for it to finish before they touch memory, so
  // they may take their places now; this one waits for the kernel before it.
  grid_launch_dependents();
  grid_dependency_wait();

  // ------------------------------------------------------------ this lane's share of a stage's copies
  const uint32_t ring = smem_addr(smem) + static_cast<uint32_t>(warp * D) * L::kSlot;
  const int64_t k_first = kbeg + ks * 16;
  // codes: rows lane / 4 and lane / 4 + 8, 32 columns each; N is a multiple of 64
  const bool c_ok = col0 + (lane & 3) * 32 < p.N;
  const uint8_t* c_src = p.codes + (k_first + (lane >> 2)) * (p.N / 2) + col0 / 2 + (lane & 3) * 16;
  const uint32_t c_dst = (lane >> 2) * kMvCodePitch + (lane & 3) * 16;
  // scales: row 4t' + i goes to place 4i + t', so that the four t of one i read 128 contiguous bytes
  const bool s_ok = col0 + (lane & 1) * 64 < p.N;
  const float* s_src = p.scales + (k_first + (lane >> 1)) * (p.N / 16) + col0 / 16 + (lane & 1) * 4;
  const uint32_t s_dst = L::kScale + (((lane >> 1) & 3) * 4 + (lane >> 3)) * 32 + (lane & 1) * 16;
  // x: 16 k of a token, one or two 16-byte pieces
  const int xm = X8 ? lane : lane >> 1;
  const bool x_ok = xm < p.M && xm < MT * 8;
  const uint8_t* x_src = static_cast<const uint8_t*>(p.x) +
                         (X8 ? xm * p.K + k_first : (xm * p.K + k_first) * 2 + (lane & 1) * 16);
  const uint32_t x_dst = L::kX + (X8 ? lane * 16 : (lane >> 1) * 32 + (lane & 1) * 16);
  auto copy_stage = [&](int i, int slot) {
    const uint32_t base = ring + slot * L::kSlot;
    const int64_t k = static_cast<int64_t>(i) * kMvRows;
    if (c_ok) {
      const uint8_t* s = c_src + k * (p.N / 2);
      cp_async16(base + c_dst, s);
      cp_async16(base + c_dst + 8 * kMvCodePitch, s + 4 * p.N);
    }
    if (s_ok) cp_async16(base + s_dst, s_src + k * (p.N / 16));
    if (x_ok) cp_async16(base + x_dst, x_src + (X8 ? k : 2 * k));
    if constexpr (RCH > 0) {
      // A: row 4t' + i goes to place 2t' + (i & 1) + 8 (i >> 1), the order of the transposing load
#pragma unroll
      for (int u = 0; u < 2 * RCH / 32; ++u) {
        const int c = lane + 32 * u, row = c / (RCH / 8), q = c % (RCH / 8);
        const int col = half * RCH + 8 * q;
        const int place = 2 * (row >> 2) + (row & 1) + 8 * ((row >> 1) & 1);
        if (col < p.r)
          cp_async16(base + L::kA + place * L::kAPitch + q * 16, p.A + (k_first + k + row) * p.r + col);
      }
    }
  };

  float acc[MT][8][4];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][j][c] = 0.0f;
  float vacc[MT][RT > 0 ? RT : 1][4];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int j = 0; j < (RT > 0 ? RT : 1); ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) vacc[a][j][c] = 0.0f;

  // scales of 8-bit x: tokens g and g + 8, one per row or one per stage (64 rows)
  float xs[MT];
  auto load_xs = [&](int i) {
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      const int m = a * 8 + g;
      xs[a] = 0.0f;
      if (m < p.M) xs[a] = __ldg(p.x_scales + (p.x_block ? m * (p.K / 64) + kbeg / 64 + i : m));
    }
  };
  if (X8) load_xs(0);

  for (int i = 0; i < D - 1; ++i) {
    if (i < nst) copy_stage(i, i);
    cp_async_commit();
  }
  int slot = 0, fill = D - 1;
  for (int i = 0; i < nst; ++i) {
    cp_async_wait<D - 2>();   // stage i has landed (this lane's copies)
    __syncwarp();             // and every lane's; and every lane is done with stage i - 1
    if (i + D - 1 < nst) copy_stage(i + D - 1, fill);
    cp_async_commit();
    const uint32_t base = ring + slot * L::kSlot;
    fill = slot;
    slot = slot + 1 == D ? 0 : slot + 1;

    // x of tokens g (and g + 8), rows 4t .. 4t+3
    float x[MT][4];
    uint32_t xh[MT][2], xl[MT][2];   // the same as bf16 pairs (X8: as two-term sums)
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      if constexpr (X8) {
        const uint32_t c = lds32(base + L::kX + (a * 8 + g) * 16 + 4 * t);
        const float2 f0 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c), __NV_E4M3)));
        const float2 f1 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c >> 16), __NV_E4M3)));
        x[a][0] = f0.x * xs[a];
        x[a][1] = f0.y * xs[a];
        x[a][2] = f1.x * xs[a];
        x[a][3] = f1.y * xs[a];
        if constexpr (RCH > 0) {
          split2(x[a][0], x[a][1], xh[a][0], xl[a][0]);
          split2(x[a][2], x[a][3], xh[a][1], xl[a][1]);
        }
      } else {
        const uint2 c = lds64(base + L::kX + (a * 8 + g) * 32 + 8 * t);
        x[a][0] = bf16_lo(c.x);
        x[a][1] = bf16_hi(c.x);
        x[a][2] = bf16_lo(c.y);
        x[a][3] = bf16_hi(c.y);
        xh[a][0] = c.x;
        xh[a][1] = c.y;
      }
    }
    if (X8 && p.x_block && i + 1 < nst) load_xs(i + 1);

    if constexpr (RCH > 0) {
      if (half * RCH < p.r) {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          uint32_t a0, a1, a2, a3;
          const uint32_t at = base + L::kA + ((lane >> 4) * 8 + (lane & 7)) * L::kAPitch + (2 * j + ((lane >> 3) & 1)) * 16;
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                       : "r"(at)
                       : "memory");
#pragma unroll
          for (int a = 0; a < MT; ++a) {
            mv_mma(vacc[a][j], a0, a1, a2, a3, xh[a][0], xh[a][1]);
            if constexpr (X8) mv_mma(vacc[a][j], a0, a1, a2, a3, xl[a][0], xl[a][1]);
          }
        }
      }
    }

#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // bytes (two columns) of rows 4t .. 4t+3 of four groups of 16 columns
      uint32_t w[4];
      asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(base + (lane & 15) * kMvCodePitch + h * 32 + (lane >> 4) * 16)
                   : "memory");
      float4 s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = lds128(base + L::kScale + (4 * k + t) * 32 + h * 16);
      uint32_t b[MT][4][2];
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        float2 u[4], v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[k] = mul2(make_float2(s[k].x, s[k].y), x[a][k]);
          v[k] = mul2(make_float2(s[k].z, s[k].w), x[a][k]);
        }
        b[a][0][0] = pack_bf16x2(u[0].x, u[1].x);
        b[a][0][1] = pack_bf16x2(u[2].x, u[3].x);
        b[a][1][0] = pack_bf16x2(u[0].y, u[1].y);
        b[a][1][1] = pack_bf16x2(u[2].y, u[3].y);
        b[a][2][0] = pack_bf16x2(v[0].x, v[1].x);
        b[a][2][1] = pack_bf16x2(v[2].x, v[3].x);
        b[a][3][0] = pack_bf16x2(v[0].y, v[1].y);
        b[a][3][1] = pack_bf16x2(v[2].y, v[3].y);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // 0x43nn is 128 + nn in bf16 (nn < 16), so minus 136 (0x4308) is code - 8
        const uint32_t lo = w[q] & 0x0F0F0F0Fu, hi = (w[q] >> 4) & 0x0F0F0F0Fu;
        const uint32_t a0 = sub_bf16x2(__byte_perm(lo, 0x43434343u, 0x4140), 0x43084308u);
        const uint32_t a1 = sub_bf16x2(__byte_perm(hi, 0x43434343u, 0x4140), 0x43084308u);
        const uint32_t a2 = sub_bf16x2(__byte_perm(lo, 0x43434343u, 0x4342), 0x43084308u);
        const uint32_t a3 = sub_bf16x2(__byte_perm(hi, 0x43434343u, 0x4342), 0x43084308u);
#pragma unroll
        for (int a = 0; a < MT; ++a) mv_mma(acc[a][4 * h + q], a0, a1, a2, a3, b[a][q][0], b[a][q][1]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();   // every ring is free: V and the partial tiles take its place

  // ------------------------------------------------------------ V of this CTA's rows, times B
  constexpr int TOK = MT * 8;
  float* Vs = reinterpret_cast<float*>(smem);                        // [4][2 RCH][TOK]
  float* part = reinterpret_cast<float*>(smem + L::kVs);             // [4][M][256]
  if constexpr (RCH > 0) {
    if (half * RCH < p.r) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          float* d = Vs + (ks * 2 * RCH + half * RCH + 16 * j + g) * TOK + a * 8 + 2 * t;
          *reinterpret_cast<float2*>(d) = make_float2(vacc[a][j][0] * p.scale, vacc[a][j][1] * p.scale);
          *reinterpret_cast<float2*>(d + 8 * TOK) = make_float2(vacc[a][j][2] * p.scale, vacc[a][j][3] * p.scale);
        }
    }
    __syncthreads();
    // the groups 2 ks and 2 ks + 1 of this warp's half, 16 adapter rows at a time
    for (int j0 = 0; j0 < p.r; j0 += 16) {
      uint32_t bw[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = j0 + 2 * t + (u & 1) + 8 * (u >> 1);
          const int64_t col = col0 + (2 * ks + q) * 16 + 2 * g;
          bw[q][u] = row < p.r && col < p.N ? __ldg(reinterpret_cast<const uint32_t*>(p.B + row * p.N + col)) : 0u;
        }
      uint32_t vh[MT][2], vl[MT][2];
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = j0 + 2 * t + (u & 1) + 8 * (u >> 1);
          v[u] = 0.0f;
          if (row < p.r) {
            const float* src = Vs + row * TOK + a * 8 + g;
            v[u] = (src[0] + src[2 * RCH * TOK]) + (src[4 * RCH * TOK] + src[6 * RCH * TOK]);
          }
        }
        split2(v[0], v[1], vh[a][0], vl[a][0]);
        split2(v[2], v[3], vh[a][1], vl[a][1]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t a0 = __byte_perm(bw[q][0], bw[q][1], 0x5410), a1 = __byte_perm(bw[q][0], bw[q][1], 0x7632);
        const uint32_t a2 = __byte_perm(bw[q][2], bw[q][3], 0x5410), a3 = __byte_perm(bw[q][2], bw[q][3], 0x7632);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j == ks) {   // the accumulators of these groups, without indexing registers
              mv_mma(acc[a][2 * j + q], a0, a1, a2, a3, vh[a][0], vh[a][1]);
              mv_mma(acc[a][2 * j + q], a0, a1, a2, a3, vl[a][0], vl[a][1]);
            }
      }
    }
  }

  // ------------------------------------------------------------ parts: 4 row steps, then the splits
  // D of a group: column 2g (c[0], c[1]) and 2g + 1 (c[2], c[3]), tokens 2t and 2t + 1
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int m = a * 8 + 2 * t + q;
      if (m < p.M) {
        float* d = part + (ks * p.M + m) * kMvTile + half * 128 + 2 * g;
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<float2*>(d + 16 * j) = make_float2(acc[a][j][q], acc[a][j][2 + q]);
      }
    }
  __syncthreads();
  // Groups of four values: Y's [M][256], then (first tile, V wanted) V's [M][r].  CTA o
  // of the cluster owns the groups [o cap, (o + 1) cap): every split pushes its sum of
  // a group into the owner's slot for it, and the owner adds the slots in split order.
  const int S = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int gy = p.M * (kMvTile / 4);
  const int groups = gy + (RCH > 0 && tile == 0 && p.V ? p.M * p.r / 4 : 0);
  const int cap = (groups + S - 1) / S;
  const uint32_t recv_addr = smem_addr(recv);
  for (int q = tid; q < groups; q += kMvThreads) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q < gy) {
      const float4* src = reinterpret_cast<const float4*>(part) + q;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float4 u = src[s * gy];
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
    } else if constexpr (RCH > 0) {
      const int e = 4 * (q - gy), m = e / p.r, j = e % p.r;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float* src = Vs + (s * 2 * RCH + j) * TOK + m;
        v.x += src[0];
        v.y += src[TOK];
        v.z += src[2 * TOK];
        v.w += src[3 * TOK];
      }
    }
    const int o = q / cap, at = q - o * cap;
    st_shared_cluster_v4(mapa_shared(recv_addr + static_cast<uint32_t>((rank * cap + at) * 16), o), v);
  }
  cluster_sync();   // every push of every split has landed
  for (int at = tid; at < cap && rank * cap + at < groups; at += kMvThreads) {
    const int q = rank * cap + at;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < S; ++s) {
      const float4 u = reinterpret_cast<const float4*>(recv)[s * cap + at];
      y.x += u.x;
      y.y += u.y;
      y.z += u.z;
      y.w += u.w;
    }
    const uint2 o = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    if (q < gy) {
      const int m = q / (kMvTile / 4);
      const int64_t col = static_cast<int64_t>(tile) * kMvTile + (q % (kMvTile / 4)) * 4;
      if (col < p.N) *reinterpret_cast<uint2*>(p.Y + m * p.N + col) = o;
    } else {
      *reinterpret_cast<uint2*>(p.V + 4 * (q - gy)) = o;   // V is (M, r), dense
    }
  }
}

// Clusters of each size a device holds at once, for one kernel variant (zero: it
// cannot run); queried once per device.
struct MvFit {
  bool done = false;
  int max_active[kMvMaxCluster + 1] = {};
};

template <int MT, int RCH, bool X8>
const MvFit& mv_fit() {
  static std::mutex mu;
  static MvFit fits[64];
  static const MvFit none{};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::lock_guard<std::mutex> lock(mu);
  MvFit& f = fits[dev];
  if (f.done) return f;
  auto fn = matvec_kernel<MT, RCH, X8>;
  constexpr uint32_t bytes = MvLayout<MT, RCH, X8>::kSmem;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess ||
      cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();
    return none;
  }
  for (int S = 1; S <= kMvMaxCluster; ++S) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1, S);
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = S;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&f.max_active[S], fn, &cfg) != cudaSuccess) f.max_active[S] = 0;
  }
  cudaGetLastError();
  f.done = true;
  return f;
}

// Splits S and rows per split: the fewest waves x (stages of a CTA + the ends).
bool mv_plan(int64_t K, int64_t N, const MvFit& fit, int& S, int64_t& Kc) {
  const int64_t tiles = (N + kMvTile - 1) / kMvTile, stages = K / kMvRows;
  int64_t best = -1;
  for (int s = 1; s <= kMvMaxCluster && s <= stages; ++s) {
    if (fit.max_active[s] < 1) continue;
    const int64_t per = (stages + s - 1) / s;
    if ((stages + per - 1) / per != s) continue;   // another s gives the same split
    const int64_t cost = (tiles + fit.max_active[s] - 1) / fit.max_active[s] * (per + 2);
    if (best < 0 || cost < best) {
      best = cost;
      S = s;
      Kc = per * kMvRows;
    }
  }
  return best >= 0;
}

template <int MT, int RCH, bool X8>
cudaError_t run_matvec(MvArgs a, cudaStream_t stream) {
  int S;
  if (!mv_plan(a.K, a.N, mv_fit<MT, RCH, X8>(), S, a.Kc)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + kMvTile - 1) / kMvTile), static_cast<unsigned>(S));
  cfg.blockDim = dim3(kMvThreads);
  cfg.dynamicSmemBytes = MvLayout<MT, RCH, X8>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = static_cast<unsigned>(S);
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  timing_before(QLORA_KERNEL_MATVEC, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, matvec_kernel<MT, RCH, X8>, a);
  timing_after(QLORA_KERNEL_MATVEC, stream);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int MT, int RCH>
cudaError_t run_by_x(const MvArgs& a, cudaStream_t stream) {
  return a.x_scales ? run_matvec<MT, RCH, true>(a, stream) : run_matvec<MT, RCH, false>(a, stream);
}

template <int MT>
cudaError_t run_by_rank(const MvArgs& a, cudaStream_t stream) {
  if (a.r == 0) return run_by_x<MT, 0>(a, stream);
  if (a.r <= 32) return run_by_x<MT, 16>(a, stream);
  if (a.r <= 64) return run_by_x<MT, 32>(a, stream);
  if (a.r <= 128) return run_by_x<MT, 64>(a, stream);
  return run_by_x<MT, 128>(a, stream);
}

}  // namespace

cudaError_t launch_matvec(const WeightView& w, const ActView& x, const uint16_t* A, const uint16_t* B, int64_t M,
                          int r, float scale, uint16_t* Y, uint16_t* V, cudaStream_t stream) {
  if (w.fmt != kFmtInt16 || M < 1 || M > kGemvMaxTokens) return cudaErrorInvalidValue;
  const MvArgs a{w.codes, w.dq_scales, x.x, x.scales, x.block, A, B, static_cast<int>(M), r, scale, w.in, w.out, 0,
                 Y, V};
  return M <= 8 ? run_by_rank<1>(a, stream) : run_by_rank<2>(a, stream);
}

}  // namespace qlora
