// The gated block's forward for few rows (M <= 128): serving and short prompts.
//
// Few rows leave the weights as the work: 0.52 bytes a weight to stream, one
// decode each, so every SM should stream and decode an equal share of both
// weights, whatever their shape, and each weight once.
//
// gated_rows_kernel.  The columns of both weights are cut into groups of 256
// (of one weight each), the K rows into steps of 64; a last group holds both
// adapters' A (64 columns each), whose "weights" need no decode.  The units
// (group, step), group by group, are dealt out in equal runs to one CTA per
// SM.  One thread streams a run's packed 64 x 128 bytes a unit by TMA through
// a ring of its own, and X's steps [rows x 64] through another (a TMA box is
// about 1 us away, longer than a unit takes, while the decoded stages, 32 KB
// each, are few); 24 decoder warps, in three turns, decode a unit's 64 x 256
// weights into shared memory as the MN-major A operand (two M = 128 products;
// the decoded tile layout of the fused GEMM), X's step is the K-major B operand
// with N = the rows rounded up to 16.  The sums D[column][row] stay in TMEM
// until the run leaves the group (a segment of the run): then four warps, which
// otherwise load and decode the scales, write them to the workspace, one slot
// per (CTA, group).  Two warps issue the products, each one half (128 columns) of
// every unit, its K slices in turn into two accumulators: a product waits 117
// clocks for the one before it on the same accumulator (29 with four in turn).
// (Neither warp may leave units out: a ring's parity cannot tell the phase before
// the last from the next.)
//
// gated_join_kernel adds a column's slots in CTA order (so the result does not
// depend on timing), forms Z = bf16(c X A) from the last group's slots (bf16 as in
// the layer: the operand that the backward's dB takes), adds
// Z·B, applies the activation and writes H (and what the backward keeps).
//
// Bound: the decode.  A row of 64 weights takes about 217 operations of the pipe
// that has the byte permutes, logic and conversions (64 lanes a clock): 870
// clocks a unit, against 512 for its 32 KB to and from shared memory and 370 for
// its 8.4 KB from HBM at 6.5 TB/s over 148 SMs.  Measured: a unit about 1020 clocks,
// that pipe 71 % busy over the launch (M = 16, 8192 x 22016, 98 us and the join 5;
// 204 MB, 2.1 TB/s) and 50 % with the start and the end of one token's 37 units a
// CTA (4096 x 11008, 34 us with the join).  Shifts as products on the other pipe
// changed nothing; a table in shared memory instead of the permutes would cost
// that the 32 KB's bandwidth.
#include "act.cuh"
#include "common.cuh"
#include "fused.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "rank.cuh"
#include "tmap.cuh"

namespace qnf4 {
namespace {

constexpr int kRwStages = 3;                      // decoded stages, one a turn
constexpr int kRwCols = 256;                      // weight columns of a group
constexpr int kRwW = kRwCols * 128;               // decoded tile: 4 x 64 rows of 128 bytes
constexpr int kRwDecWarps = 8;                    // one row of 64 weights per decoder thread and unit
constexpr int kRwTurns = 3;                       // groups of decoder warps that take units in turn
constexpr int kRwScaleWarps = 4;                  // scales, units in turn, and the segments' sums
constexpr int kRwMmaWarps = 2;
constexpr int kRwThreads = (1 + kRwMmaWarps + kRwScaleWarps + kRwDecWarps * kRwTurns) * 32;
constexpr int kRwTwoBufRows = 64;                 // up to here two segments' sums fit TMEM
constexpr int kRwLookahead = 4;                   // units whose scales go before a segment's sums
constexpr int kRwPk = 64 * 128;                   // packed bytes of a unit
constexpr int kRwPkStages = 8;                    // packed bytes and scales
constexpr int kRwMaxX = 8;                        // stages of the X ring, at most
constexpr int kRwSmemMax = 232448;                // 227 KB, the opt-in limit per CTA
constexpr int kRwMaxRows = 128;

// Roles of the 31 warps: 0 .. 3 scales and sums (warp q may read TMEM lanes
// 32q .. 32q + 31), then the two that issue products and the TMA warp, then the
// decoders, six on every scheduler (a warp's is its number modulo 4).
enum RowsRole : int { kRwMmaWarp = kRwScaleWarps, kRwTmaWarp = kRwMmaWarp + kRwMmaWarps, kRwFirstDec };

struct RowsArgs {
  int M, K, N;
  int mpad;            // rows rounded up to 16: the N of the products
  int nk;              // K-steps
  int gw;              // groups per weight
  int per;             // units per CTA
  int units;           // (2 gw + 1) nk
  int acc_cols;        // TMEM columns of an accumulator (mpad, or the power of two above it)
  int nbuf;            // segments whose sums TMEM holds: 2 (1 above 64 rows)
  int tmem_cols;       // nbuf x 2 halves x even and odd slices x acc_cols
  int x_stages;
  ScaleView sv[2];
  const uint8_t* packed[2];
  float* part;         // [slots][M][256]
  int32_t* d_status;
};

// X takes what shared memory the other rings leave, up to eight stages (three
// at 128 rows).
int rows_x_stages(int mpad) {
  const int left = kRwSmemMax - 4096 - kRwStages * kRwW - kRwPkStages * (kRwPk + 1024);
  const int n = left / (mpad * 128);
  return n < kRwMaxX ? n : kRwMaxX;
}
size_t rows_smem(int mpad) {
  return 1024 + static_cast<size_t>(kRwStages) * kRwW + static_cast<size_t>(kRwPkStages) * (kRwPk + 1024) +
         static_cast<size_t>(rows_x_stages(mpad)) * mpad * 128 + 1024 + 512;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

__device__ __forceinline__ uint4 lds128(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr));
  return v;
}

// Whether the phase with this parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A wait that is usually over at once: the abort flag is read only when not.
__device__ __forceinline__ bool rows_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || (!*abort_flag && mbar_wait(bar, parity));
}

// kNf4: both weights have the NF4 codebook.
template <bool kNf4>
__global__ void __launch_bounds__(kRwThreads, 1)
    gated_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmPg,
                      const __grid_constant__ CUtensorMap tmPu, const __grid_constant__ CUtensorMap tmAg,
                      const __grid_constant__ CUtensorMap tmAu, const RowsArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int xbytes = args.mpad * 128;
  uint8_t* sW = smem;
  uint8_t* sP = sW + kRwStages * kRwW;
  uint8_t* sX = sP + kRwPkStages * kRwPk;
  float* sS = reinterpret_cast<float*>(sX + args.x_stages * xbytes);   // scales [stage][4 blocks][64 rows]
  float* t8 = sS + kRwPkStages * 256;
  uint64_t* full = reinterpret_cast<uint64_t*>(t8 + 256);
  uint64_t* empty = full + kRwStages;
  uint64_t* pfull = empty + kRwStages;
  uint64_t* pempty = pfull + kRwPkStages;
  uint64_t* xfull = pempty + kRwPkStages;
  uint64_t* xempty = xfull + kRwMaxX;
  uint64_t* tfull = xempty + kRwMaxX;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const bool dq0 = args.sv[0].code8 != nullptr, dq1 = args.sv[1].code8 != nullptr;
  if (dq0 || dq1) build_t8(t8);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRwStages; ++s) {
      mbar_init(&full[s], kRwDecWarps);   // a turn's decoder warps
      mbar_init(&empty[s], kRwMmaWarps);
    }
    for (int s = 0; s < kRwPkStages; ++s) {
      mbar_init(&pfull[s], 2);             // the packed bytes' producer, the scale warp
      mbar_init(&pempty[s], kRwDecWarps);
    }
    for (int s = 0; s < kRwMaxX; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], kRwMmaWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], kRwMmaWarps);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kRwMmaWarp) {
    tmem_alloc(tmem_holder, static_cast<uint32_t>(args.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // wait for the preceding kernel, then let the join launch: it may then read
  // everything but this kernel's sums at once
  pdl_wait();
  pdl_launch_dependents();

  const int u0 = static_cast<int>(blockIdx.x) * args.per;
  const int u1 = min(args.units, u0 + args.per);

  if (warp == kRwTmaWarp) {
    // ---------------- TMA: packed bytes and X of every unit ----------------
    // Two rings, each refilled as soon as a stage of it is free.
    if (lane == 0) {
      tma_prefetch_desc(&tmX);
      tma_prefetch_desc(&tmPg);
      tma_prefetch_desc(&tmPu);
      const int uw = min(u1, 2 * args.gw * args.nk);   // the adapters have no packed bytes
      int pu = u0, pg = u0 / args.nk, pkk = u0 - pg * args.nk;
      int xu = u0, xkk = pkk;
      uint32_t ps = 0, pph = 1, xs = 0, xph = 1;
      uint64_t t0 = 0;
      bool ok = true;
      while (pu < uw || xu < u1) {
        bool moved = false;
        if (xu < u1 && mbar_test_wait(&xempty[xs], xph)) {
          mbar_arrive_expect_tx(&xfull[xs], static_cast<uint32_t>(xbytes));
          tma_load_2d(sX + xs * xbytes, &tmX, &xfull[xs], xkk * 64, 0);
          if (++xkk == args.nk) xkk = 0;
          ++xu;
          if (++xs == static_cast<uint32_t>(args.x_stages)) { xs = 0; xph ^= 1; }
          moved = true;
        }
        if (pu < uw && mbar_test_wait(&pempty[ps], pph)) {
          mbar_arrive_expect_tx(&pfull[ps], kRwPk);
          const bool second = pg >= args.gw;
          tma_load_2d(sP + ps * kRwPk, second ? &tmPu : &tmPg, &pfull[ps], (second ? pg - args.gw : pg) * 128,
                      pkk * 64);
          if (++pkk == args.nk) { pkk = 0; ++pg; }
          ++pu;
          if (++ps == kRwPkStages) { ps = 0; pph ^= 1; }
          moved = true;
        }
        if (moved) {
          t0 = 0;
        } else {
          __nanosleep(40);
          const uint64_t t = globaltimer_ns();
          if (t0 == 0) t0 = t;
          if (*abort_flag || t - t0 > kWaitLimitNs) { ok = false; break; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        // copies in flight land before the CTA exits: the latest of each X
        // stage (a packed stage's barrier also counts its scale warp, which may
        // have given up, so those are given the time of a copy)
        const int nx = min(xu - u0, args.x_stages);
        for (int i = 0; i < nx; ++i) {
          if (xs == 0) { xs = static_cast<uint32_t>(args.x_stages); xph ^= 1; }
          --xs;
          (void)mbar_wait(&xfull[xs], xph ^ 1);
        }
        const uint64_t t = globaltimer_ns();
        while (globaltimer_ns() - t < 1000000) __nanosleep(1000);
      }
    }
  } else if (warp >= kRwMmaWarp && warp < kRwTmaWarp) {
    // ------------------------------ MMA issuers ----------------------------
    // Warp m has half m of every unit.  The whole warp runs the loop and the
    // elected lane issues.
    const uint32_t m = static_cast<uint32_t>(warp - kRwMmaWarp);
    const uint32_t idesc = idesc_bf16_f32(128, args.mpad, 1, 0);
    const uint64_t w0 = smem_desc(smem_u32(sW) + m * 16384, 8192, 1024), x0 = smem_desc(smem_u32(sX), 16, 1024);
    const uint32_t whi = static_cast<uint32_t>(w0 >> 32), xhi = static_cast<uint32_t>(x0 >> 32);
    const uint32_t acc_cols = static_cast<uint32_t>(args.acc_cols);
    const uint32_t elected = elect_one();
    bool ok = true;
    // the adapters have one half
    const int uend = m == 0 ? u1 : min(u1, 2 * args.gw * args.nk);
    const uint32_t nx = static_cast<uint32_t>(args.x_stages);
    uint32_t s = 0, ph = 0, xs = 0, xph = 0, b = 0, tph = 1;
    int u = u0;
    for (int ub = min(u1, (u0 / args.nk + 1) * args.nk); ok; ub = min(u1, ub + args.nk)) {
      // a segment: wait until its accumulators have been read
      if (!rows_wait(&tempty[b], tph, abort_flag)) { ok = false; break; }
      const uint32_t d = tmem + (b * 2 + m) * 2 * acc_cols;
      uint32_t c = 0;
      for (; u < ub; ++u) {
        if (!rows_wait(&xfull[xs], xph, abort_flag) || !rows_wait(&full[s], ph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        if (u < uend) {
          const uint32_t wlo = static_cast<uint32_t>(w0) + s * (kRwW >> 4);
          const uint32_t xlo = static_cast<uint32_t>(x0) + xs * static_cast<uint32_t>(xbytes >> 4);
          umma_bf16_lo(elected, d, wlo, whi, xlo, xhi, idesc, c);
          umma_bf16_lo(elected, d + acc_cols, wlo + 128, whi, xlo + 2, xhi, idesc, c);
          umma_bf16_lo(elected, d, wlo + 256, whi, xlo + 4, xhi, idesc, 1u);
          umma_bf16_lo(elected, d + acc_cols, wlo + 384, whi, xlo + 6, xhi, idesc, 1u);
        }
        umma_commit_if(elected, smem_u32(&empty[s]));
        umma_commit_if(elected, smem_u32(&xempty[xs]));
        c = 1;
        if (++s == kRwStages) { s = 0; ph ^= 1; }
        if (++xs == nx) { xs = 0; xph ^= 1; }
      }
      if (!ok) break;
      umma_commit_if(elected, smem_u32(&tfull[b]));
      if (++b == static_cast<uint32_t>(args.nbuf)) { b = 0; tph ^= 1; }
      if (ub >= u1) break;
    }
    if (!ok) *abort_flag = 1;
    // every product is done before the CTA gives up its TMEM
    umma_commit_if(elected, smem_u32(&drain[m]));
    (void)mbar_wait(&drain[m], 0);
  } else if (warp < kRwScaleWarps) {
    // ---------------------------- scales and sums --------------------------
    // Scales: a'[block][row] of every weight unit into the ring; zero for blocks
    // past the weight's columns.  Lane l has block l & 3 of rows (l >> 2) + 8 i
    // and keeps the raw loads of its next unit in flight.  A segment's sums
    // come after the scales of the kRwLookahead units behind it, so that the
    // decoders do not run dry while this warp waits for the products.
    const int q = warp;
    const int uw = min(u1, 2 * args.gw * args.nk);   // the adapters have no scales
    const int nb = lane & 3, rl = lane >> 2;
    const float off0 = dq0 ? __ldg(args.sv[0].offset) : 0.0f, off1 = dq1 ? __ldg(args.sv[1].offset) : 0.0f;
    const int64_t bpr = args.N / 64;
    float v[8];
    uint32_t qc[8];
    auto load = [&](int u) {
      const int g = u / args.nk, kk = u - g * args.nk;
      const bool second = g >= args.gw;
      const int n0 = (second ? g - args.gw : g) * kRwCols + nb * 64;
      const ScaleView& sv = second ? args.sv[1] : args.sv[0];
#pragma unroll
      for (int i = 0; i < 8; ++i) { v[i] = 0.0f; qc[i] = 0u; }
      if (u < uw && n0 < args.N) {
        const int64_t blk = (static_cast<int64_t>(kk) * 64 + rl) * bpr + n0 / 64;
        if (sv.code8 == nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __ldg(sv.absmax + blk + 8 * i * bpr);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            qc[i] = __ldg(sv.code8 + blk + 8 * i * bpr);
            v[i] = __ldg(sv.s2 + ((blk + 8 * i * bpr) >> 8));
          }
        }
      }
    };
    bool ok = true;
    int us = u0 + q;                                 // this warp's next unit of scales
    uint32_t ps = static_cast<uint32_t>(q), pph = 1;
    int ua = u0, ub = min(u1, (u0 / args.nk + 1) * args.nk);   // the next segment's units
    uint32_t b = 0, tph = 0;
    load(us);
    while (ok) {
      if (us < uw && us < ub + kRwLookahead) {
        const int g = us / args.nk;
        const bool second = g >= args.gw;
        const bool dq = (second ? dq1 : dq0) && (second ? g - args.gw : g) * kRwCols + nb * 64 < args.N;
        if (!rows_wait(&pempty[ps], pph, abort_flag)) { ok = false; break; }
        float* dst = sS + ps * 256 + nb * 64 + rl;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[8 * i] = dq ? __fadd_rn(__fmul_rn(t8[qc[i]], v[i]), second ? off1 : off0) : v[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[ps]);
        us += kRwScaleWarps;
        ps += kRwScaleWarps;
        if (ps >= kRwPkStages) { ps -= kRwPkStages; pph ^= 1; }
        load(us);
      } else if (ua < u1) {
        if (!rows_wait(&tfull[b], tph, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const int g = ua / args.nk;
        const int halves = g == 2 * args.gw ? 1 : 2;
        float* dst = args.part + (static_cast<int64_t>(blockIdx.x) + g) * args.M * kRwCols + q * 32 + lane;
        for (int p = 0; p < halves; ++p) {
          for (int m0 = 0; m0 < args.mpad; m0 += 16) {
            uint32_t x[16], y[16];
            const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>((b * 2 + p) * 2 * args.acc_cols + m0);
            __syncwarp();
            tmem_ld_32x32b_x16(at, x);
            tmem_ld_32x32b_x16(at + static_cast<uint32_t>(args.acc_cols), y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (m0 + i < args.M)
                dst[static_cast<int64_t>(m0 + i) * kRwCols + p * 128] =
                    __uint_as_float(x[i]) + __uint_as_float(y[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[b]);
        if (++b == static_cast<uint32_t>(args.nbuf)) { b = 0; tph ^= 1; }
        ua = ub;
        ub = min(u1, ub + args.nk);
      } else {
        break;
      }
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ------------------------------- decoders ------------------------------
    const int id = warp - kRwFirstDec;
    const int turn = id / kRwDecWarps, wi = id % kRwDecWarps;   // a turn's warps two on each scheduler
    // eight lanes of a load or store phase hold eight rows of one block (no
    // bank conflict under the swizzles)
    const int kr = wi * 8 + (lane & 7), nb = lane >> 3;
    // this thread's row in the turn's decoded stage (its 16-byte chunks in
    // swizzled order), and in stage 0 of the packed ring
    const uint32_t row = smem_u32(sW) + turn * kRwW + nb * 8192 + kr * 128 + ((kr & 7) << 4);
    const uint32_t pk0 = smem_u32(sP) + kr * 128 + (((nb * 2) ^ (kr & 7)) << 4);
    const float* const sc0 = sS + nb * 64 + kr;
    const int uw = min(u1, 2 * args.gw * args.nk);
    uint64_t* const wfull = &full[turn];
    uint64_t* const wempty = &empty[turn];
    bool ok = true;
    uint32_t ph = 1;
    uint32_t ps = static_cast<uint32_t>(turn), pph = 0;
    int u = u0 + turn;
#pragma unroll 1
    for (; u < uw; u += kRwTurns) {
      if (!rows_wait(&pfull[ps], pph, abort_flag)) { ok = false; break; }
      const uint32_t src = pk0 + ps * kRwPk;
      const uint4 p0 = lds128(src), p1 = lds128(src ^ 16u);
      const float a = sc0[ps * 256];
      uint32_t H[4], L[4];
      if constexpr (kNf4)
        build_lut_nf4(a, H, L);
      else
        build_lut(kNF4g + 16 * (u >= args.gw * args.nk ? args.sv[1].codebook : args.sv[0].codebook), a, H, L);
      if (!rows_wait(wempty, ph, abort_flag)) { ok = false; break; }
      const uint32_t pw[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
      for (uint32_t c = 0; c < 8; ++c) sts128(row ^ (c << 4), decode8(pw[c], H, L));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(wfull);
        mbar_arrive(&pempty[ps]);
      }
      ph ^= 1;
      ps += kRwTurns;
      if (ps >= kRwPkStages) { ps -= kRwPkStages; pph ^= 1; }
    }
    // the adapters' A: one thread of a turn lets TMA bring both tiles
#pragma unroll 1
    for (; ok && u < u1; u += kRwTurns) {
      if (!rows_wait(wempty, ph, abort_flag)) { ok = false; break; }
      if (lane == 0) {
        if (wi == 0) {
          const int k0 = (u - 2 * args.gw * args.nk) * 64;
          uint8_t* dst = sW + turn * kRwW;
          mbar_arrive_expect_tx(wfull, 16384u);
          tma_load_2d(dst, &tmAg, wfull, 0, k0);
          tma_load_2d(dst + 8192, &tmAu, wfull, 0, k0);
        } else {
          mbar_arrive(wfull);
        }
      }
      __syncwarp();
      ph ^= 1;
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) raise_status(args.d_status, QLORA_ERR_TIMEOUT);
  if (warp == kRwMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(args.tmem_cols));
  }
}

// ---------------------------------------------------------------------------
// Join: a block has 64 columns (a lane two of them) and kJoinTok rows.  Its
// eight warps first take the rank in eight slices for Z·B (each lane's loads of
// B, which no earlier kernel of the call writes, all in flight at once), then
// one row each: the sum of the slices, the column's slots, the activation.
// ---------------------------------------------------------------------------
constexpr int kJoinTok = 8;
constexpr int kJoinWarps = 8;

struct JoinArgs {
  int M, N, r;
  int nk, gw, per;
  const float* part;
  const uint16_t *Bg, *Bu;
  float c;
  int act;
  uint16_t* H;
  GatedKept kept;
  int32_t* d_status;
};

// The sum over a group's slots at `off`, in CTA order.
__device__ __forceinline__ float2 slot_sum2(const JoinArgs& a, int g, int64_t off) {
  const int c0 = static_cast<int>(static_cast<int64_t>(g) * a.nk / a.per);
  const int c1 = static_cast<int>((static_cast<int64_t>(g + 1) * a.nk - 1) / a.per);
  const int64_t slot = static_cast<int64_t>(a.M) * kRwCols;
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float2 v = *reinterpret_cast<const float2*>(a.part + (c + g) * slot + off);
    s.x += v.x;
    s.y += v.y;
  }
  return s;
}

__global__ void __launch_bounds__(kJoinWarps * 32)
    gated_join_kernel(const JoinArgs a) {
  __shared__ float zs[2][kJoinTok][64];
  __shared__ float2 red[kJoinWarps][2][kJoinTok][32];   // [slice][g, u][row][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * 64 + 2 * lane;   // N is a multiple of 64: always inside
  const int t0 = blockIdx.y * kJoinTok;
  const int nt = min(kJoinTok, a.M - t0);
  pdl_launch_dependents();
  // rank slice of this warp: rows warp, warp + 8, ... of B
  uint32_t bg[8], bu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = warp + 8 * i;
    bg[i] = bu[i] = 0;
    if (j < a.r) {
      bg[i] = __ldg(reinterpret_cast<const uint32_t*>(a.Bg + static_cast<int64_t>(j) * a.N + n));
      bu[i] = __ldg(reinterpret_cast<const uint32_t*>(a.Bu + static_cast<int64_t>(j) * a.N + n));
    }
  }
  pdl_wait();
  // this thread's row and columns: the slots of g and u
  float2 g2 = make_float2(0.0f, 0.0f), u2 = g2;
  if (warp < nt) {
    const int64_t off = static_cast<int64_t>(t0 + warp) * kRwCols + (n & (kRwCols - 1));
    g2 = slot_sum2(a, n / kRwCols, off);
    u2 = slot_sum2(a, a.gw + n / kRwCols, off);
  }
  // Z of the block's rows: element e = (row, adapter, two ranks)
  for (int e = threadIdx.x; e < nt * 64; e += kJoinWarps * 32) {
    const int t = e >> 6, w = (e >> 5) & 1, j = (e & 31) * 2;
    float2 z = make_float2(0.0f, 0.0f);
    if (j < a.r) z = slot_sum2(a, 2 * a.gw, static_cast<int64_t>(t0 + t) * kRwCols + w * 64 + j);
    const uint32_t zb = pack_bf16x2(a.c * z.x, a.c * z.y);
    zs[w][t][j] = j < a.r ? __uint_as_float(zb << 16) : 0.0f;
    zs[w][t][j + 1] = j + 1 < a.r ? __uint_as_float(zb & 0xFFFF0000u) : 0.0f;
    if (blockIdx.x == 0 && a.kept.Zg != nullptr) {
      uint16_t* dst = (w == 0 ? a.kept.Zg : a.kept.Zu) + static_cast<int64_t>(t0 + t) * a.r;
      if (j < a.r) dst[j] = static_cast<uint16_t>(zb);
      if (j + 1 < a.r) dst[j + 1] = static_cast<uint16_t>(zb >> 16);
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kJoinTok; ++t) {
    if (t < nt) {
      float2 sg = make_float2(0.0f, 0.0f), su = sg;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = warp + 8 * i;
        if (j < a.r) {
          const float zg = zs[0][t][j], zu = zs[1][t][j];
          sg.x = fmaf(zg, __uint_as_float(bg[i] << 16), sg.x);
          sg.y = fmaf(zg, __uint_as_float(bg[i] & 0xFFFF0000u), sg.y);
          su.x = fmaf(zu, __uint_as_float(bu[i] << 16), su.x);
          su.y = fmaf(zu, __uint_as_float(bu[i] & 0xFFFF0000u), su.y);
        }
      }
      red[warp][0][t][lane] = sg;
      red[warp][1][t][lane] = su;
    }
  }
  __syncthreads();
  if (warp >= nt) return;
#pragma unroll
  for (int s = 0; s < kJoinWarps; ++s) {
    const float2 x = red[s][0][warp][lane], y = red[s][1][warp][lane];
    g2.x += x.x;
    g2.y += x.y;
    u2.x += y.x;
    u2.y += y.y;
  }
  const int64_t row = t0 + warp;
  const int64_t at = row * a.N + n;
  *reinterpret_cast<uint32_t*>(a.H + at) =
      act_mul2(a.act, g2.x, g2.y, u2.x, u2.y);
  if (a.kept.G != nullptr) {
    *reinterpret_cast<uint32_t*>(a.kept.G + at) = pack_bf16x2(g2.x, g2.y);
    *reinterpret_cast<uint32_t*>(a.kept.U + at) = pack_bf16x2(u2.x, u2.y);
  }
  if (a.kept.G8 != nullptr) {
    // the warp's 64 columns are one block of the checkpoint
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float x0 = round_bf16(w == 0 ? g2.x : u2.x), x1 = round_bf16(w == 0 ? g2.y : u2.y);
      float amax = fmax_nan(fabsf(x0), fabsf(x1));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
      const float s = act8_scale(amax), inv = act8_inverse(s);
      const uint32_t x[1] = {w == 0 ? pack_bf16x2(g2.x, g2.y) : pack_bf16x2(u2.x, u2.y)};
      uint32_t q[2];
      act8_round(x, s, inv, q);
      *reinterpret_cast<uint16_t*>((w == 0 ? a.kept.G8 : a.kept.U8) + at) =
          static_cast<uint16_t>(__byte_perm(q[0], q[1], 0x0040));
      if (lane == 0) {
        (w == 0 ? a.kept.Gs : a.kept.Us)[row * (a.N / 64) + n / 64] = s;
        if (!(amax <= FLT_MAX)) raise_status(a.d_status, QLORA_ERR_NONFINITE);
      }
    }
  }
}

struct RowsPlan {
  int gw, nk, units, per, ctas;
};

// Equal runs of units over one CTA per SM of the sizing count (at least two
// units a CTA: a unit alone is less than its start-up).
RowsPlan rows_plan(int64_t K, int64_t N) {
  RowsPlan p;
  p.gw = static_cast<int>((N + kRwCols - 1) / kRwCols);
  p.nk = static_cast<int>(K / 64);
  p.units = (2 * p.gw + 1) * p.nk;
  p.per = (p.units + g_ws_sms - 1) / g_ws_sms;
  if (p.per < 2) p.per = 2;
  p.ctas = (p.units + p.per - 1) / p.per;
  return p;
}

}  // namespace

bool gated_rows_fit(int64_t M, int64_t K, int64_t N) {
  return M <= kRwMaxRows && (2 * ((N + kRwCols - 1) / kRwCols) + 1) * (K / 64) < (1ll << 30);
}

size_t gated_rows_workspace_bytes(int64_t M, int64_t K, int64_t N, int r) {
  const RowsPlan p = rows_plan(K, N);
  const int rp = padded_rank(r);
  return align256(static_cast<size_t>(p.ctas + 2 * p.gw + 1) * M * kRwCols * 4) +
         (rp != r ? 2 * align256(static_cast<size_t>(K) * rp * 2) : 0);
}

cudaError_t launch_gated_rows(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                              const GatedWeights& w, uint16_t* H, const GatedKept& kept, void* ws,
                              size_t ws_bytes, int32_t* d_status, cudaStream_t st) {
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  const RowsPlan p = rows_plan(K, N);
  const int rp = padded_rank(r);
  float* part = static_cast<float*>(cur.take(static_cast<size_t>(p.ctas + 2 * p.gw + 1) * M * kRwCols * 4));
  const uint16_t *Ag = w.Ag, *Au = w.Au;
  cudaError_t e = cudaSuccess;
  if (rp != r) {
    uint16_t* Apg = static_cast<uint16_t*>(cur.take(static_cast<size_t>(K) * rp * 2));
    uint16_t* Apu = static_cast<uint16_t*>(cur.take(static_cast<size_t>(K) * rp * 2));
    if (!cur.ok) return cudaErrorInvalidValue;
    e = launch_pad_sets(PadSet{{w.Ag, w.Au}, {Apg, Apu}, {K, K}}, 2, r, rp, st);
    if (e != cudaSuccess) return e;
    Ag = Apg;
    Au = Apu;
  }
  if (!cur.ok) return cudaErrorInvalidValue;
  static DeviceOnce once;
  e = once.run([](int) {
    const int most = kRwSmemMax;
    cudaError_t a = cudaFuncSetAttribute(gated_rows_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return a != cudaSuccess ? a
                            : cudaFuncSetAttribute(gated_rows_kernel<true>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  RowsArgs a{};
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.mpad = static_cast<int>((M + 15) / 16 * 16);
  a.nk = p.nk;
  a.gw = p.gw;
  a.per = p.per;
  a.units = p.units;
  a.nbuf = a.mpad <= kRwTwoBufRows ? 2 : 1;
  a.acc_cols = 16;
  while (a.acc_cols < a.mpad) a.acc_cols *= 2;
  a.tmem_cols = a.nbuf * 4 * a.acc_cols;
  a.x_stages = rows_x_stages(a.mpad);
  a.sv[0] = w.sv_g;
  a.sv[1] = w.sv_u;
  a.packed[0] = w.packed_g;
  a.packed[1] = w.packed_u;
  a.part = part;
  a.d_status = d_status;
  CUtensorMap tX, tPg, tPu, tAg, tAu;
  if (!make_tmap_2d(&tPg, w.packed_g, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, N / 2, N / 2, 128, 64, kSW128))
    return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tPu, w.packed_u, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, N / 2, N / 2, 128, 64, kSW128))
    return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tX, X, kBF16, 2, M, K, K, 64, a.mpad, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tAg, Ag, kBF16, 2, K, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tAu, Au, kBF16, 2, K, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  {
    ProfScope prof(kProfGated, st);
    const bool nf4 = w.sv_g.codebook == QLORA_CODEBOOK_NF4 && w.sv_u.codebook == QLORA_CODEBOOK_NF4;
    e = launch_pdl(nf4 ? gated_rows_kernel<true> : gated_rows_kernel<false>, dim3(static_cast<unsigned>(p.ctas)), dim3(kRwThreads),
                   rows_smem(a.mpad), st, 1, tX, tPg, tPu, tAg, tAu, a);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  JoinArgs j{};
  j.M = a.M;
  j.N = a.N;
  j.r = r;
  j.nk = p.nk;
  j.gw = p.gw;
  j.per = p.per;
  j.part = part;
  j.Bg = w.Bg;
  j.Bu = w.Bu;
  j.c = w.c;
  j.act = w.act;
  j.H = H;
  j.kept = kept;
  j.d_status = d_status;
  {
    ProfScope prof(kProfGated, st);
    e = launch_pdl(gated_join_kernel,
                   dim3(static_cast<unsigned>(N / 64), static_cast<unsigned>((M + kJoinTok - 1) / kJoinTok)),
                   dim3(kJoinWarps * 32), 0, st, 1, j);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qnf4
