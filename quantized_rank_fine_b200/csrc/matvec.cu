// A few tokens (M <= 16) through a weight of 4-bit integers with one scale per 16:
//
//   Y[m][n] = sum_k x[m][k] q[k][n] s[k][n / 16] + sum_j V[m][j] B[j][n],  V = scale X A
//
// Its floor is to read the codes and scales once (0.75 B a weight); what it is bound by
// is below.
//
//   * Split over K without a second pass: both terms are linear in the rows, so a
//     CTA that owns the rows [k0, k0 + Kc) of a column tile forms x W of its
//     rows and also V of its rows times B; the parts of a tile are added over a
//     thread-block cluster in split order.  One launch, no scratch, no atomics.
//   * Stages of 8 KB of codes, 4 KB of scales, x and A come by TMA through a shared
//     ring; eight warps consume them: 128 columns x 16 rows each at up to 8 tokens,
//     64 columns x 32 rows above.  The warps take turns at issuing the copies (a
//     warp of its own for that would leave 96 registers a thread instead of 128).
//   * Tensor cores with the weight as the 16 x 16 A operand and 8 tokens as the B
//     operand: mma.sync m16n8k16 (128-row tcgen05 tiles have no use for 16 tokens).
//     The 16 operand rows are the 16 columns that share a scale, so the scale
//     folds into x: B = x s, and A is the integer q itself, exact in bf16.
//     The byte transpose of ldmatrix (m16n16 .b8) hands lane (g, t) one byte, two
//     columns, of four rows; a byte permute sets the nibble into bf16 128 + code
//     and one packed subtraction of 136 leaves q.
//   * x s goes in as two bf16 terms, bf16(x s) and bf16 of what that leaves: 16 bits, so a
//     product is within 2^-16 of itself and the output's own rounding decides the error,
//     at every size of the weight.  (One term is within 2^-8: the relative error against
//     64 bits is then 0.0024 instead of 0.0017, an output formed by cancellation is off by
//     2^-8 of its products, and the time 12 to 30% less: 4096 x 4096, rank 16, 1 token
//     7.1 against 7.9 us, 4096 x 11008, 16 tokens 17.5 against 24.0.  TF32 products, 11
//     bits, take the time of two bf16 terms.)  V, too, is a sum of two bf16 numbers; sums
//     are fp32.
//
// Measured (graph of calls over weights larger than L2): 4096 x 11008 with rank 16 at 1,
// 4 and 16 tokens 15.9, 16.1 and 23.7 us (2.2, 2.1 and 1.5 TB/s); 4096 x 4096 8.1, 8.6 and
// 11.7 us.  47 warp-instructions for each 16 x 16 weights at 1 token, 72 at 16 (whole
// launch); 55% of the cycles issue one, DRAM runs at 21 and 15% of its peak and the tensor
// pipe at 20 and 28%: bound by the instructions that unpack, scale and split with 16
// warps an SM, then by the ends of a launch (3 us for the smallest weight).
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

#include <cudaTypedefs.h>

#include <mutex>

namespace qlora {

namespace {

using namespace sm100;

constexpr int kMvWarps = 8;                      // KS row groups x NC column groups
constexpr int kMvThreads = kMvWarps * 32;
constexpr int kMvWeights = 16384;                // weights of a stage: 64 rows of 256 columns or 128 of 128
constexpr int kMvMaxCluster = 16;

struct MvArgs {
  const float* x_scales;
  int x_block;
  const uint16_t* B;
  int M, r;
  float scale;
  int64_t K, N;
  int64_t Kc;             // rows per split (multiple of 64)
  uint16_t* Y;
  uint16_t* V;            // saved V, or nullptr
  uint32_t* status;
};

enum : int { kXBf16 = 0, kXRow = 1, kXBlock = 2 };

// TW: columns of a CTA.  MT: token tiles of 8.  RC: adapter columns held (0: no
// adapter; 16, 64, 128, 256).  XM: x in bf16, or in E4M3 codes with one scale a row or
// one per 64 columns.
template <int TW, int MT, int RC, int XM>
struct MvLayout {
  static constexpr bool X8 = XM != kXBf16;
  static constexpr int kTok = MT * 8;
  static constexpr int kRows = kMvWeights / TW;                     // rows a stage
  // columns of a warp: wide where the accumulators allow it, as x is unpacked once for all of them
  static constexpr int kCols = MT == 1 ? 128 : 64;
  static constexpr int kNC = TW / kCols;
  static constexpr int kKS = kMvWarps / kNC;                        // warps that share the rows of a stage
  static constexpr int kSteps = kRows / 16 / kKS;                   // 16-row steps of a warp in a stage
  static constexpr int kGroups = kCols / 16;
  static constexpr int kOwn = TW / 16 / kMvWarps;                   // groups whose adapter term a warp adds
  // a stage, as TMA writes it, each tile swizzled by its row length (32, 64 or 128
  // bytes): codes (TW / 2 bytes a row), x (64 k of a token a row), scales (TW / 4), A
  // (boxes of 16 columns, or of 64)
  static constexpr int kCodePieces = TW / 32, kScalePieces = TW / 64;
  static constexpr uint32_t kX = 8192;
  static constexpr uint32_t kXPitch = X8 ? 64 : 128;
  static constexpr uint32_t kXBox = kTok * kXPitch;
  static constexpr uint32_t kScale = kX + kRows / 64 * kXBox;
  static constexpr uint32_t kA = (kScale + 4096 + 1023) / 1024 * 1024;
  static constexpr int kABox = RC < 64 ? RC : 64;                   // columns a box
  static constexpr uint32_t kABytes = kRows * kABox * 2;
  static constexpr uint32_t kStage = (kA + kRows * RC * 2 + 1023) / 1024 * 1024;
  // after the loop: V of the row groups (fp32), V as two bf16 terms, the partial tiles
  static constexpr int kPartPitch = TW + 4;                         // floats a row of a partial tile
  static constexpr int kVPitch = kTok + 4;
  static constexpr int kWPitch = RC + 8;
  // one adapter tile: the column groups take the row steps in turn, and each warp has a V of its own
  static constexpr bool kTurns = RC == 16 && kNC > 1;
  static constexpr int kVs = kTurns ? kMvWarps : kKS;
  static constexpr uint32_t kW = kVs * RC * kVPitch * 4;
  static constexpr uint32_t kPart = kW + (RC ? 2 * kTok * kWPitch * 2 : 0);
  static constexpr uint32_t kTail = kPart + kKS * kTok * kPartPitch * 4;
  static constexpr uint32_t kRecv = (kTok * TW / 4 + kTok * RC / 4 + kMvMaxCluster) * 16;
  static constexpr uint32_t bytes(int depth) {   // + 1 KB to align the ring to the swizzle atom
    return 1024 + (depth * kStage > kTail ? depth * kStage : kTail) + kRecv;
  }
  static constexpr int depth(uint32_t budget) {
    int d = 6;
    while (d > 2 && bytes(d) > budget) --d;
    return d;
  }
  // two CTAs on an SM where that leaves three stages each, else one
  static constexpr int kCtas = bytes(3) <= 113 * 1024 ? 2 : 1;
  static constexpr int kDepth = depth(kCtas == 2 ? 113 * 1024 : 226 * 1024);
  static constexpr uint32_t kSmem = bytes(kDepth);
  // adapter tiles of 16 columns a warp multiplies: kNC j + its column group
  static constexpr int kRT = (RC / 16 + kNC - 1) / kNC;
};

// Byte offset of 16-byte piece c of row `row` in a TMA tile of n pieces a row with the
// swizzle of its row length (2, 4 or 8 pieces: 32, 64 or 128 bytes).
template <int n>
__device__ __forceinline__ uint32_t piece(int row, int c) {
  constexpr int shift = n == 2 ? 2 : (n == 4 ? 1 : 0);
  return static_cast<uint32_t>(row * (n * 16) + ((c ^ ((row >> shift) & (n - 1))) << 4));
}

#define QLORA_MV_MMA                                                                                             \
  "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"    \
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                            \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1)
// In the loop, where its result is carried round, the compiler may place it among the
// loads; after the loop it stays where it is, outside of any lane's branch.
__device__ __forceinline__ void mv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm(QLORA_MV_MMA);
}
__device__ __forceinline__ void mv_mma_here(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(QLORA_MV_MMA);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two binary32 numbers in one 64-bit register, and their product by one instruction.
__device__ __forceinline__ uint64_t twice(float a) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ float2 mul2(uint64_t a, uint64_t b) {
  float2 d;
  asm("{\n\t.reg .b64 p;\n\tmul.rn.f32x2 p, %2, %3;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "l"(a), "l"(b));
  return d;
}

// bf16(v) and bf16(v - bf16(v)) of two values, packed: together 16 bits of each.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(v0, v1);
  lo = pack_bf16x2(v0 - bf16_lo(hi), v1 - bf16_hi(hi));
}

template <int TW, int MT, int RC, int XM>
__global__ void __launch_bounds__(kMvThreads, (MvLayout<TW, MT, RC, XM>::kCtas))
matvec_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scales,
              const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_a, const MvArgs p) {
  using L = MvLayout<TW, MT, RC, XM>;
  constexpr bool X8 = L::X8, blocked = XM == kXBlock;
  constexpr int D = L::kDepth, RT = L::kRT, TOK = L::kTok, NC = L::kNC, KS = L::kKS, G = L::kGroups;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset, not through an integer: the compiler then knows a shared address
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* recv = smem + (L::kSmem - 1024 - L::kRecv);
  __shared__ __align__(8) uint64_t bars[2 * D];
  const uint32_t full0 = smem_addr(bars), empty0 = smem_addr(bars + D);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int ks = warp % KS, cg = warp / KS;   // row group and column group of the warp
  const int tile = blockIdx.x, split = blockIdx.y;
  const int64_t kbeg = split * p.Kc;
  // rows past K read as zeros: a half last stage adds nothing
  const int nst = static_cast<int>(((p.K - kbeg < p.Kc ? p.K - kbeg : p.Kc) + L::kRows - 1) / L::kRows);
  const int64_t col0 = static_cast<int64_t>(tile) * TW + cg * L::kCols;   // first column of this warp

  cluster_started_arrive();
  if (tid == 0) {
    for (int s = 0; s < D; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, kMvWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_codes);
    tma_prefetch_desc(&tm_scales);
    tma_prefetch_desc(&tm_x);
    if (RC > 0) tma_prefetch_desc(&tm_a);
  }
  __syncthreads();
  // The kernels after this one wait for it to finish before they touch memory, so
  // they may take their places now; this one waits for the kernel before it.
  grid_launch_dependents();
  grid_dependency_wait();

  // The copies of stage i into slot s (one lane).
  auto issue = [&](int i, int s) {
    const uint32_t bytes = 8192 + 4096 + L::kRows * RC * 2 + L::kRows / 64 * static_cast<uint32_t>(p.M) * L::kXPitch;
    const uint32_t dst = smem_addr(smem + s * L::kStage), bar = full0 + 8 * s;
    const int32_t k = static_cast<int32_t>(kbeg + static_cast<int64_t>(i) * L::kRows);
    mbar_arrive_expect_tx(bar, bytes);
    tma_load_2d(dst, &tm_codes, bar, tile * (TW / 2), k);
    tma_load_2d(dst + L::kScale, &tm_scales, bar, tile * (TW / 16), k);
#pragma unroll
    for (int c = 0; c < L::kRows / 64; ++c) tma_load_2d(dst + L::kX + c * L::kXBox, &tm_x, bar, k + 64 * c, 0);
#pragma unroll
    for (int c = 0; c < RC; c += 64) tma_load_2d(dst + L::kA + (c / 64) * L::kABytes, &tm_a, bar, c, k);
  };
  if (tid == 0)
    for (int i = 0; i < D && i < nst; ++i) issue(i, i);

  float acc[MT][G][4];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][j][c] = 0.0f;
  float vacc[MT][RT > 0 ? RT : 1][4];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int j = 0; j < (RT > 0 ? RT : 1); ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) vacc[a][j][c] = 0.0f;

  // The scales of x and B may have been written by the kernel in front while this one
  // was already resident, so they are read by ordinary loads behind the wait, never by
  // the read-only path.  (Past L1 the block scales, eight blocks of a token to a sector,
  // come from L2 at every stage: 4096 x 11008, rank 16, 4 tokens 23.9 us against 18.1.)
  //
  // Scales of 8-bit x.  One a row: the loop multiplies with the codes alone, exact in
  // bf16, and the finished sums are scaled.  One per 64 rows: those of tokens g and
  // g + 8 (a warp's rows of a stage lie in one block of 64).
  const int64_t nblk = p.K / 64;
  float xs[MT];
  auto load_xs = [&](int i) {
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      const int64_t m = a * 8 + g < p.M ? a * 8 + g : 0;   // a column past M is never stored
      const int64_t blk = kbeg / 64 + L::kRows / 64 * i + ks * L::kSteps / 4;
      xs[a] = p.x_scales[m * nblk + (blk < nblk ? blk : 0)];
    }
  };
  if constexpr (blocked) load_xs(0);

  // B of 16 adapter rows and this warp's groups of columns (kOwn ks, ... of its columns).
  // With one token tile the first are loaded here, so that nothing waits for them after
  // the loop (4096 x 4096, 1 token: 7.8 -> 7.4 us); two token tiles have no registers
  // left for that (they spilled: 19.2 -> 23.3 us at 4096 x 11008 with block scales).
  constexpr int OWN = L::kOwn;
  const int64_t bcol = col0 + 16 * OWN * ks + 2 * g;
  constexpr int CH = RC < 64 ? 1 : 4;   // at a time
  uint32_t bw[CH][OWN][4] = {};
  auto load_b = [&](int i, int j0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = j0 + 2 * t + (u & 1) + 8 * (u >> 1);
      const bool in = row < p.r && bcol < p.N;   // N is a multiple of 64: a warp's groups lie inside or outside
#pragma unroll
      for (int o = 0; o < OWN; ++o)
        bw[i][o][u] = in ? *reinterpret_cast<const uint32_t*>(p.B + row * p.N + bcol + 16 * o) : 0u;
    }
  };
  if constexpr (RC > 0 && MT == 1) load_b(0, 0);

  // The lane's rows of a 16-row step are 4t + (i ^ (t >> 1)), i = 0 .. 3: with the swizzles
  // above, the four lanes' scales of one i then lie on different banks, and so do the
  // eight code rows of each phase of the transposing load.
  const uint32_t base0 = smem_addr(smem);
  const int flip = t >> 1;
  const int r0 = ks * 16 * L::kSteps;                                  // first row of this warp in a stage
  const int wrow = (lane & 12) + ((lane & 3) ^ ((lane >> 3) & 1));     // ldmatrix: row 4t' + i of the codes
  const int ta = (lane & 7) >> 1;                                      // ... and 2t' + (i & 1) of A
  const int arow = 4 * ta + (((lane & 1) + 2 * (lane >> 4)) ^ (ta >> 1));
  // offsets in a stage; 16 rows on, they grow by whole rows of each tile
  uint32_t w_off[G / 4], s_off[G / 4][4], a_off[RT > 0 ? RT : 1];
#pragma unroll
  for (int j = 0; j < G / 4; ++j) {
    w_off[j] = piece<L::kCodePieces>(r0 + wrow, cg * (G / 2) + 2 * j + (lane >> 4));
#pragma unroll
    for (int k = 0; k < 4; ++k) s_off[j][k] = L::kScale + piece<L::kScalePieces>(r0 + 4 * t + (k ^ flip), cg * (G / 4) + j);
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int tr = NC * j + cg;
    a_off[j] = L::kA + (RC == 16 ? piece<2>(r0 + arow, (lane >> 3) & 1)
                                 : (tr / 4) * L::kABytes + piece<8>(r0 + arow, 2 * (tr & 3) + ((lane >> 3) & 1)));
  }
  // Not unrolled over the ring: constant slot addresses save some adds (4096 x 11008, 1
  // token, no adapter: 11.2 against 11.7 us), but six copies of the body come in from
  // memory at every launch (4096 x 4096: 6.9 against 5.9).
  int s = 0;
  uint32_t ph = 0;
  bool ok = true;   // a wait that gave up raises the status word; the rest then runs through quickly
#pragma unroll 1
  for (int i = 0; i < nst; ++i) {
    // refill the slot of the stage before the last one, which every warp is done with by now or soon
    constexpr int kBack = 2;
    if (i >= kBack && i - kBack + D < nst && warp == (i & (kMvWarps - 1)) && lane == 0) {
      const int old = s >= kBack ? s - kBack : s - kBack + D;
      ok = mbar_wait_limit(empty0 + 8 * old, s >= kBack ? ph : ph ^ 1u, p.status, kFlagTimeoutProducer,
                           ok ? kWaitLimitNs : 1000000u) && ok;
      issue(i - kBack + D, old);
    }
    ok = mbar_wait_limit(full0 + 8 * s, ph, p.status, kFlagTimeoutMma, ok ? kWaitLimitNs : 1000000u) && ok;
    __syncwarp();
    const uint8_t* at = smem + s * L::kStage;
    const uint32_t base = base0 + s * L::kStage;
    float xs_now[MT];
#pragma unroll
    for (int a = 0; a < MT; ++a) xs_now[a] = blocked ? xs[a] : 1.0f;
    if (blocked && i + 1 < nst) load_xs(i + 1);

#pragma unroll
    for (int h = 0; h < L::kSteps; ++h) {   // 16-row steps
      const int kstep = ks * L::kSteps + h;
      // x of tokens g (and g + 8) at the lane's rows
      float x[MT][4];
      uint32_t xb[MT][2];   // bf16 x: the pairs as they are
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        const int m = a * 8 + g;
        if constexpr (X8) {
          uint32_t c = *reinterpret_cast<const uint32_t*>(at + L::kX + (kstep / 4) * L::kXBox + piece<4>(m, kstep & 3) + 4 * t);
          c = __byte_perm(c, 0u, flip ? 0x2301 : 0x3210);
          const float2 f0 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c), __NV_E4M3)));
          const float2 f1 =
              __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(c >> 16), __NV_E4M3)));
          x[a][0] = f0.x;
          x[a][1] = f0.y;
          x[a][2] = f1.x;
          x[a][3] = f1.y;
          if constexpr (blocked) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[a][k] *= xs_now[a];
          }
        } else {
          const uint2 c = *reinterpret_cast<const uint2*>(
              at + L::kX + (kstep / 4) * L::kXBox + piece<8>(m, 2 * (kstep & 3) + (t >> 1)) + 8 * (t & 1));
          xb[a][0] = __byte_perm(c.x, 0u, flip ? 0x1032 : 0x3210);
          xb[a][1] = __byte_perm(c.y, 0u, flip ? 0x1032 : 0x3210);
          x[a][0] = bf16_lo(xb[a][0]);
          x[a][1] = bf16_hi(xb[a][0]);
          x[a][2] = bf16_lo(xb[a][1]);
          x[a][3] = bf16_hi(xb[a][1]);
        }
      }

      if constexpr (RC > 0) {
        if (L::kTurns ? (i * L::kSteps + h) % NC == cg : 16 * cg < p.r) {
          uint32_t xh[MT][2], xl[MT][2];   // x for the adapter: exact, or (with block scales) a sum of two bf16 terms
#pragma unroll
          for (int a = 0; a < MT; ++a) {
            if constexpr (X8) {
              xh[a][0] = pack_bf16x2(x[a][0], x[a][1]);
              xh[a][1] = pack_bf16x2(x[a][2], x[a][3]);
              if constexpr (blocked) {
                split2(x[a][0], x[a][1], xh[a][0], xl[a][0]);
                split2(x[a][2], x[a][3], xh[a][1], xl[a][1]);
              }
            } else {
              xh[a][0] = xb[a][0];
              xh[a][1] = xb[a][1];
            }
          }
#pragma unroll
          for (int j = 0; j < RT; ++j) {
            if (L::kTurns || 16 * (NC * j + cg) < p.r) {   // tile NC j + cg of 16 adapter columns
              uint32_t a0, a1, a2, a3;
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                           : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                           : "r"(base + a_off[j] + h * 16 * (RC == 16 ? 32 : 128)));
#pragma unroll
              for (int a = 0; a < MT; ++a) {
                mv_mma(vacc[a][j], a0, a1, a2, a3, xh[a][0], xh[a][1]);
                if constexpr (blocked) mv_mma(vacc[a][j], a0, a1, a2, a3, xl[a][0], xl[a][1]);
              }
            }
          }
        }
      }

      uint64_t xx[MT][4];
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int k = 0; k < 4; ++k) xx[a][k] = twice(x[a][k]);
#pragma unroll
      for (int j = 0; j < G / 4; ++j) {   // four groups of 16 columns at a time
        // bytes (two columns) of the lane's rows
        uint32_t w[4];
        asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(base + w_off[j] + h * 16 * (TW / 2)));
        ulonglong2 sc[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[k] = *reinterpret_cast<const ulonglong2*>(at + s_off[j][k] + h * 16 * (TW / 4));
        uint32_t b[MT][4][2], bl[MT][4][2];   // x s as bf16 pairs, and what they leave over
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          float2 u[4], v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            u[k] = mul2(sc[k].x, xx[a][k]);
            v[k] = mul2(sc[k].y, xx[a][k]);
          }
          auto fold = [&](int q, float k0, float k1, float k2, float k3) {
            split2(k0, k1, b[a][q][0], bl[a][q][0]);
            split2(k2, k3, b[a][q][1], bl[a][q][1]);
          };
          fold(0, u[0].x, u[1].x, u[2].x, u[3].x);
          fold(1, u[0].y, u[1].y, u[2].y, u[3].y);
          fold(2, v[0].x, v[1].x, v[2].x, v[3].x);
          fold(3, v[0].y, v[1].y, v[2].y, v[3].y);
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
          for (int a = 0; a < MT; ++a) {
            mv_mma(acc[a][4 * j + q], a0, a1, a2, a3, b[a][q][0], b[a][q][1]);
            mv_mma(acc[a][4 * j + q], a0, a1, a2, a3, bl[a][q][0], bl[a][q][1]);
          }
        }
      }
    }
    __syncwarp();   // every lane is done with the stage
    if (lane == 0) mbar_arrive(empty0 + 8 * s);
    if (++s == D) {
      s = 0;
      ph ^= 1u;
    }
  }

  // ------------------------------------------------------------ V of this CTA's rows, times B
  float* Vs = reinterpret_cast<float*>(smem);                                // [kVs][ranks][kVPitch]
  uint16_t* W = reinterpret_cast<uint16_t*>(smem + L::kW);                   // [2 terms][tok][kWPitch]
  float* part = reinterpret_cast<float*>(smem + L::kPart);                   // [KS][tok][L::kPartPitch]
  if constexpr (RC > 0) {
#pragma unroll
    for (int i = MT == 1 ? 1 : 0; i < CH; ++i) load_b(i, 16 * i);
    __syncthreads();   // every ring is free
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int tr = L::kTurns ? 0 : 16 * (NC * j + cg);
      if (tr < p.r) {
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          float* d = Vs + ((L::kTurns ? warp : ks) * RC + tr + g) * L::kVPitch + a * 8 + 2 * t;
          *reinterpret_cast<float2*>(d) = make_float2(vacc[a][j][0] * p.scale, vacc[a][j][1] * p.scale);
          *reinterpret_cast<float2*>(d + 8 * L::kVPitch) = make_float2(vacc[a][j][2] * p.scale, vacc[a][j][3] * p.scale);
        }
      }
    }
    __syncthreads();
    const int r16 = (p.r + 15) & ~15;
    for (int e = tid; e < r16 * TOK; e += kMvThreads) {
      const int j = e / TOK, m = e % TOK;
      float v = 0.0f;
      if (j < p.r)
#pragma unroll
        for (int k = 0; k < L::kVs; ++k) v += Vs[(k * RC + j) * L::kVPitch + m];
      uint32_t hi, lo;
      split2(v, 0.0f, hi, lo);
      W[m * L::kWPitch + j] = static_cast<uint16_t>(hi);
      W[(TOK + m) * L::kWPitch + j] = static_cast<uint16_t>(lo);
    }
    __syncthreads();
    for (int j0 = 0; j0 < p.r; j0 += 16 * CH) {
      if (j0 > 0) {
#pragma unroll
        for (int i = 0; i < CH; ++i) load_b(i, j0 + 16 * i);
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int j = j0 + 16 * i;
        if (j < p.r) {
          uint32_t b4[OWN][4];
#pragma unroll
          for (int o = 0; o < OWN; ++o) {
            b4[o][0] = __byte_perm(bw[i][o][0], bw[i][o][1], 0x5410);
            b4[o][1] = __byte_perm(bw[i][o][0], bw[i][o][1], 0x7632);
            b4[o][2] = __byte_perm(bw[i][o][2], bw[i][o][3], 0x5410);
            b4[o][3] = __byte_perm(bw[i][o][2], bw[i][o][3], 0x7632);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint32_t* vh = reinterpret_cast<const uint32_t*>(W + (m * 8 + g) * L::kWPitch + j + 2 * t);
            const uint32_t* vl = vh + TOK * L::kWPitch / 2;
#pragma unroll
            for (int q = 0; q < G; ++q)
              if (q / OWN == ks) {   // the accumulators of these groups, without indexing registers
                const uint32_t(&w)[4] = b4[q % OWN];
                mv_mma_here(acc[m][q], w[0], w[1], w[2], w[3], vh[0], vh[4]);
                mv_mma_here(acc[m][q], w[0], w[1], w[2], w[3], vl[0], vl[4]);
              }
          }
        }
      }
    }
  } else {
    __syncthreads();   // every ring is free
  }

  // ------------------------------------------------------------ parts: the row groups, then the splits
  // D of a group: column 2g (c[0], c[1]) and 2g + 1 (c[2], c[3]), tokens 2t and 2t + 1
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int m = a * 8 + 2 * t + q;
      if (m < p.M) {
        float* d = part + (ks * TOK + m) * L::kPartPitch + cg * L::kCols + 2 * g;
#pragma unroll
        for (int j = 0; j < G; ++j) *reinterpret_cast<float2*>(d + 16 * j) = make_float2(acc[a][j][q], acc[a][j][2 + q]);
      }
    }
  __syncthreads();
  // Groups of four values: Y's [M][TW], then (first tile, V wanted) V's [M][r].  CTA o
  // of the cluster owns the groups [o cap, (o + 1) cap): every split pushes its sum of
  // a group into the owner's slot for it, and the owner adds the slots in split order.
  const int S = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int gy = p.M * (TW / 4);
  const int groups = gy + (RC > 0 && tile == 0 && p.V ? p.M * p.r / 4 : 0);
  const int cap = (groups + S - 1) / S;
  const uint32_t recv_addr = smem_addr(recv);
  cluster_started_wait();
  for (int q = tid; q < groups; q += kMvThreads) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q < gy) {
      const float* src = part + (q / (TW / 4)) * L::kPartPitch + 4 * (q % (TW / 4));
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const float4 u = *reinterpret_cast<const float4*>(src + k * TOK * L::kPartPitch);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
    } else {
      const int e = 4 * (q - gy), m = e / p.r;
#pragma unroll
      for (int k = 0; k < L::kVs; ++k) {
        const float* src = Vs + (k * RC + e % p.r) * L::kVPitch + m;
        v.x += src[0];
        v.y += src[L::kVPitch];
        v.z += src[2 * L::kVPitch];
        v.w += src[3 * L::kVPitch];
      }
    }
    if constexpr (XM == kXRow) {   // the scales of the rows
      const float f = p.x_scales[q < gy ? q / (TW / 4) : 4 * (q - gy) / p.r];
      v.x *= f;
      v.y *= f;
      v.z *= f;
      v.w *= f;
    }
    const int o = q / cap, to = q - o * cap;
    st_shared_cluster_v4(mapa_shared(recv_addr + static_cast<uint32_t>((rank * cap + to) * 16), o), v);
  }
  cluster_sync();   // every push of every split has landed
  for (int to = tid; to < cap && rank * cap + to < groups; to += kMvThreads) {
    const int q = rank * cap + to;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < S; ++s) {
      const float4 u = reinterpret_cast<const float4*>(recv)[s * cap + to];
      y.x += u.x;
      y.y += u.y;
      y.z += u.z;
      y.w += u.w;
    }
    const uint2 o = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    if (q < gy) {
      const int m = q / (TW / 4);
      const int64_t col = static_cast<int64_t>(tile) * TW + (q % (TW / 4)) * 4;
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

template <int TW, int MT, int RC, int XM>
const MvFit& mv_fit() {
  static std::mutex mu;
  static MvFit fits[64];
  static const MvFit none{};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return none;
  std::lock_guard<std::mutex> lock(mu);
  MvFit& f = fits[dev];
  if (f.done) return f;
  auto fn = matvec_kernel<TW, MT, RC, XM>;
  constexpr uint32_t bytes = MvLayout<TW, MT, RC, XM>::kSmem;
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

// Splits S and rows per split of a tile width, and its cost: waves x (stages of a CTA +
// the ends of a CTA, about three).  -1 if no cluster size fits.
int64_t mv_plan(int64_t K, int64_t N, int tw, const MvFit& fit, int& S, int64_t& Kc) {
  const int64_t rows = kMvWeights / tw, tiles = (N + tw - 1) / tw, stages = (K + rows - 1) / rows;
  int64_t best = -1;
  for (int s = 1; s <= kMvMaxCluster && s <= stages; ++s) {
    if (fit.max_active[s] < 1) continue;
    const int64_t per = (stages + s - 1) / s;
    if ((stages + per - 1) / per != s) continue;   // another s gives the same split
    const int64_t cost = (tiles + fit.max_active[s] - 1) / fit.max_active[s] * (per + 3);
    if (best < 0 || cost < best) {
      best = cost;
      S = s;
      Kc = per * rows;
    }
  }
  return best;
}

PFN_cuTensorMapEncodeTiled_v12000 mv_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {   // looked up once, whichever threads call first
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(
        e == cudaSuccess && q == cudaDriverEntryPointSuccess ? ptr : nullptr);
  }();
  return fn;
}

// Row-major (rows x cols) of `type` with elements of `size` bytes; a box of
// box_cols x box_rows, swizzled by its row length (32, 64 or 128 bytes).
bool mv_map(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, int64_t rows, int64_t cols,
            int box_cols, int box_rows) {
  auto enc = mv_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * size)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  const int row = box_cols * size;
  const CUtensorMapSwizzle swizzle = row == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                                     : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                 : CU_TENSOR_MAP_SWIZZLE_128B;
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the tensor maps are made of.
struct MvInputs {
  const uint8_t* codes;
  const float* scales;
  const void* x;
  const uint16_t* A;
};

template <int TW, int MT, int RC, int XM>
cudaError_t run_matvec(MvArgs a, int S, const MvInputs& in, cudaStream_t stream) {
  using L = MvLayout<TW, MT, RC, XM>;
  CUtensorMap tc, ts, tx, ta;
  if (!mv_map(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, in.codes, a.K, a.N / 2, TW / 2, L::kRows) ||
      !mv_map(&ts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, in.scales, a.K, a.N / 16, TW / 16, L::kRows) ||
      !(L::X8 ? mv_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, in.x, a.M, a.K, 64, a.M)
           : mv_map(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, in.x, a.M, a.K, 64, a.M)) ||
      (RC > 0 && !mv_map(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, in.A, a.K, a.r, L::kABox, L::kRows)))
    return cudaErrorInvalidValue;
  if (RC == 0) ta = tx;   // not read
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + TW - 1) / TW), static_cast<unsigned>(S));
  cfg.blockDim = dim3(kMvThreads);
  cfg.dynamicSmemBytes = L::kSmem;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, matvec_kernel<TW, MT, RC, XM>, tc, ts, tx, ta, a);
  timing_after(QLORA_KERNEL_MATVEC, stream);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The tile width is the one of lower cost: 128 columns make twice the tiles of half the
// clusters, which fill the device better where N gives few tiles (11008 x 4096, 4
// tokens, rank 16: 15.8 us against 17.3 with 256 before the second term).  On a tie 128
// columns, whose smaller clusters spread more evenly and end sooner (5120 x 5120, 16
// tokens, rank 16: 16.7 us against 20.6; 1024 x 1024: 5.2 against 5.6; 4096 x 11008: 24.0
// against 23.7), but 256 with an adapter of more than 64 columns, which is then read half
// as often (rank 256, 16 tokens: 512 x 512 14.1 us against 16.9, 5120 x 5120 29.6 against
// 47.6; rank 64: 7.3 against 7.5 at 1024 x 1024, 24.0 against 19.8 at 5120 x 5120).
template <int MT, int RC, int XM>
cudaError_t run_by_width(MvArgs a, const MvInputs& in, cudaStream_t stream) {
  int S1 = 0, S2 = 0;
  int64_t k1 = 0, k2 = 0;
  const int64_t c1 = mv_plan(a.K, a.N, 128, mv_fit<128, MT, RC, XM>(), S1, k1);
  const int64_t c2 = mv_plan(a.K, a.N, 256, mv_fit<256, MT, RC, XM>(), S2, k2);
  if (c1 < 0 && c2 < 0) return cudaErrorInvalidValue;
  if (c2 < 0 || (c1 >= 0 && (RC > 64 ? c1 < c2 : c1 <= c2))) {
    a.Kc = k1;
    return run_matvec<128, MT, RC, XM>(a, S1, in, stream);
  }
  a.Kc = k2;
  return run_matvec<256, MT, RC, XM>(a, S2, in, stream);
}

template <int MT, int RC>
cudaError_t run_by_x(const MvArgs& a, const MvInputs& in, cudaStream_t stream) {
  if (!a.x_scales) return run_by_width<MT, RC, kXBf16>(a, in, stream);
  return a.x_block ? run_by_width<MT, RC, kXBlock>(a, in, stream) : run_by_width<MT, RC, kXRow>(a, in, stream);
}

template <int MT>
cudaError_t run_by_rank(const MvArgs& a, const MvInputs& in, cudaStream_t stream) {
  if (a.r == 0) return run_by_x<MT, 0>(a, in, stream);
  if (a.r <= 16) return run_by_x<MT, 16>(a, in, stream);
  if (a.r <= 64) return run_by_x<MT, 64>(a, in, stream);
  if (a.r <= 128) return run_by_x<MT, 128>(a, in, stream);
  return run_by_x<MT, 256>(a, in, stream);
}

}  // namespace

cudaError_t launch_matvec(const WeightView& w, const ActView& x, const uint16_t* A, const uint16_t* B, int64_t M,
                          int r, float scale, uint16_t* Y, uint16_t* V, uint32_t* status, cudaStream_t stream) {
  if (w.fmt != kFmtInt16 || M < 1 || M > kGemvMaxTokens) return cudaErrorInvalidValue;
  const MvArgs a{x.scales, x.block, B, static_cast<int>(M), r, scale, w.in, w.out, 0, Y, V, status};
  const MvInputs in{w.codes, w.dq_scales, x.x, A};
  return M <= 8 ? run_by_rank<1>(a, in, stream) : run_by_rank<2>(a, in, stream);
}

}  // namespace qlora
