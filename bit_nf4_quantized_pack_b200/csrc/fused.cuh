// The fused NF4-decode GEMM on sm_100a, shared by the layer (linear.cu) and the
// operators built on it (gated.cu, loss.cu).  Every translation unit that
// includes this file gets its own copy of what it uses.
#pragma once

#include <math_constants.h>

#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "tmap.cuh"

namespace qnf4 {
namespace {

// code values of the two codebooks: [0, 16) NF4, [16, 32) uniform INT4
__constant__ float kNF4g[32] = {QNF4_TABLE_VALUES, QNF4_INT4_VALUES};

// ===========================================================================
// Fused NF4-decode GEMM.  kMode:
//   kModeFwd        Y = X·Ŵ + Zc·B
//   kModeBwd        dX = G·Ŵᵀ + dZ·Aᵀ
//   kModeGatedFwd   g = X·Ŵg + Zg·Bg and u = X·Ŵu + Zu·Bu side by side, H = act(g)·u
//   kModeGatedBwd   dX = dG·Ŵgᵀ + dU·Ŵuᵀ + dZg·Agᵀ + dZu·Auᵀ
//   kModeLossStats  the maximum and sum of exponentials of each row of X·Ŵ over
//                   256 columns, and the label's logit
//   kModeLossGrad   P = bf16(softmax(X·Ŵ) - onehot) over a piece of columns
//   kModeLossDX     dX (+)= dloss·(P·Ŵᵀ) over a piece of columns
// "forward" and "backward" below are the operand layouts: the modes with Ŵᵀ
// (Bwd, GatedBwd, LossDX) use the backward one.
//
// Persistent pairs of CTAs on neighbouring SMs (a 1 x 2 thread-block cluster)
// run CTA-pair tensor-core products (tcgen05.mma.cta_group::2, M = 256,
// N = 256, K = 16), issued by CTA rank 0 for both: the A operand is split by
// rows (128 per CTA) and the B operand by columns (128 per CTA), each half in
// its own CTA's shared memory, and each CTA's TMEM receives its 128 rows of D
// over all 256 columns.  So each CTA stages only half of each operand, and
// the tensor core reads 8 KB of shared memory per CTA and 16-wide K slice
// for a 128 x 256 x 16 product per SM.
//   forward   pair tile 512 rows x 256 columns; CTA q holds rows
//             m0 + 256q + [0, 256) (slices h = 0, 1 of 128 rows, the K-major
//             A operand of accumulator h) and decodes columns n0 + 128q + [0,
//             128) of every weight K-step (the MN-major B operand);
//   backward  transposed: pair tile 256 output columns x 512 dY rows; CTA q
//             decodes the weight rows n0 + 128q + [0, 128) (the K-major A
//             operand: its output columns) and holds dY rows m0 + 256h + 128q +
//             [0, 128) (its half of the B operand of accumulator h = 0, 1).
// TMEM: two accumulators of 128 lanes x 256 fp32 columns per CTA (all 512).
//
// Shared memory holds two rings per CTA.  Activation tiles (256 x 64 bf16,
// K-major, two TMA boxes of 128 rows) have 4 stages; TMA loads of both CTAs
// complete on CTA 0's barrier (the cta_group::2 form of the copy), which CTA
// 0's producer arms with both CTAs' bytes.  Decoded weight tiles have 4
// stages; decoder warps write them as 128 rows of 128 bytes, each row one NF4
// block of 64 consecutive weights (row R at R*128, 16-byte chunk c at
// (c ^ (R & 7))*16, the 128-byte swizzle pattern):
//   forward   row R = 64*nb + k: weights (k0+k, n0+128q+64nb .. +63) — an
//             MN-major operand (atoms of 8 k-rows x 64 n; 8 KB between
//             n-atoms);
//   backward  row R: weights (n0+128q+R, k0 .. k0+63) of W, i.e. row R of
//             Ŵᵀ's K-major operand.
// Each decoder thread owns one row and loads its 32 packed bytes and its
// block scale straight from global memory K-steps ahead; both CTAs' decoder
// warps arrive on CTA 0's barrier of the stage.  The MMA's commit releases
// the stages and signals the accumulators in both CTAs (multicast), and both
// CTAs' epilogue warps release an accumulator on CTA 0's barrier.
//
// After the last K-step of a tile the LoRA step (the gated modes' first before the
// last two, see lora_early) takes two activation stages: Zc (or dZ) as the
// activation tile and B (or A) as the weight tile, both by TMA with the rank
// padded to a multiple of 16 by TMA's zero fill; the decoder warps skip it.  The
// epilogue releases each accumulator as soon as it has read it, so the next tile's
// first MMAs overlap the drain of the last; until then they wait for it, so its
// eight warps only lay their rows out in shared memory, from where TMA stores them
// (store_rows).  In the backward a warp's TMEM load gives each lane one output
// column over 32 consecutive rows.
//
// Bound: the tensor pipe, 1025 clocks a K-step of a full pair tile (1024 for its
// products) where the decode keeps up, then the waves of tiles and the power cap.
// Tiles of 256 rows are bound by the decode's latency (about 950 clocks a
// K-step).  Measured at 4096^3: forward 95 us, dX 105 beside dA and dB, 1375
// TFLOP/s a launch.
//
// The gated forward is the forward with another meaning of the 256 columns of
// a pair tile: CTA 0 decodes 128 columns of the gate weight, CTA 1 the same
// 128 columns of the up weight, so a row's g and u meet in one thread of the
// epilogue and the decode per product stays that of one weight.  Its two LoRA
// steps give each CTA the rows of its own B and zeros (a box past the
// matrix's last row) in the other's step.  The gated backward runs through
// the K-steps of dG·Ŵgᵀ and then of dU·Ŵuᵀ in the same accumulators.
// Where dX has few tiles (few rows), a tile's K-steps are cut into `splits`
// equal items; each leaves fp32 sums of its own, which split_join_kernel adds in
// order.  The first item of a tile has its LoRA steps.
// These modes and the loss's split activation rows as m0 + 256h + 128q and
// leave out slice h = 1 where a tile has no more than 256 rows.
// ===========================================================================
enum FusedMode : int {
  kModeFwd = 0,
  kModeBwd = 1,
  kModeGatedFwd = 2,
  kModeGatedBwd = 3,
  kModeLossStats = 4,
  kModeLossGrad = 5,
  kModeLossDX = 6
};
constexpr bool mode_transposed(int m) { return m == kModeBwd || m == kModeGatedBwd || m == kModeLossDX; }
constexpr bool mode_gated(int m) { return m == kModeGatedFwd || m == kModeGatedBwd; }
constexpr bool mode_loss(int m) { return m >= kModeLossStats; }
constexpr int mode_lora_steps(int m) { return mode_loss(m) ? 0 : (mode_gated(m) ? 2 : 1); }
// dX modes may split the contraction of a tile over several work items
constexpr bool mode_splits(int m) { return m == kModeGatedBwd || m == kModeLossDX; }
constexpr int mode_tile_cols(int m) { return m == kModeGatedFwd ? 128 : 256; }

constexpr int kFAStages = 4;          // activation tiles (TMA)
constexpr int kFBStages = 4;          // decoded weight tiles (decoder warps)
constexpr int kFBN = 128;             // decoded rows per CTA and K-step
constexpr int kFSlices = 2;           // 128-row activation slices per CTA = accumulators
constexpr int kFAccCols = 256;        // TMEM columns per accumulator (the pair MMA's N)
constexpr int kFPairRows = 512;       // activation rows of a pair tile
constexpr int kFPairCols = 256;       // output columns of a pair tile
constexpr int kFA = kFSlices * 128 * 128;   // 256 x 64 bf16
constexpr int kFB = kFBN * 128;             // 128 x 64 bf16
constexpr int kFDecWarps = kFBN / 32;       // one weight-tile row per decoder thread and K-step
// Decoder groups of kFDecWarps warps take turns by K-step (group g decodes the
// steps g, g + kFDecGroups, ...), so each warp has kFDecGroups K-steps of time
// per row and its loads reach further ahead.
constexpr int kFDecGroups = 2;
constexpr int kFDecAll = kFDecWarps * kFDecGroups;
// Epilogue warps: four would cover the 128 lanes of TMEM; of eight each has half
// of the columns, since an accumulator that is being drained holds up the next
// tile's products.
constexpr int kFEpiWarps = 8;
constexpr int kFThreads = (2 + kFDecAll + kFEpiWarps) * 32;  // TMA, MMA, decoders, epilogue
// The epilogue's staging: per warp a ring of kFOutSlots tiles of 32 rows x 64 bytes.
constexpr int kFOutSlots = 2;
constexpr int kFOutSlot = 32 * 64;
constexpr int kFOut = kFEpiWarps * kFOutSlots * kFOutSlot;
constexpr size_t kFSmem = 1024 + kFAStages * kFA + kFBStages * kFB + kFOut + 1024 + 512;
static_assert(kFSlices * kFAccCols == 512 && kFBN == 128, "accumulators fill TMEM");
static_assert(kFSmem <= 232448, "fused kernel shared memory");

struct FusedArgs {
  int M;          // rows of the activation / output
  int Nout;       // output columns (forward: N, backward: K; loss: columns of the piece)
  int Nw;         // row length of the weight (N); blocks per weight row = Nw/64
  int nk;         // K-steps over the contraction (forward: K/64, backward: N/64)
  int rsteps;     // MMAs of K=16 in a LoRA step (ceil(r/16))
  int m_tiles, n_tiles;
  ScaleView sv;
  const uint8_t* packed;
  int32_t* d_status;
};

// Tile shape of the operators' modes, and the split contraction of the dX modes: K-steps per item (steps * splits >= nk),
// and with splits > 1 the items' sums [splits][M][Nout].
struct SplitArgs : FusedArgs {
  int rows;       // activation rows of a tile: 512 or 256
  int splits, steps;
  float* part;
};

// What the gated modes need besides: the second weight (nk counts the K-steps
// of both in the backward), and in the forward the activation and the buffers
// that keep g and u for the backward (all null: nothing is kept).
struct GatedArgs : SplitArgs {
  ScaleView sv2;
  const uint8_t* packed2;
  int act;
  int keep;             // 0: nothing; 1: g and u in bf16; 2: in 8 bits, scales [M][Nout/64]
  float *Gs, *Us;
};

// What the loss modes need besides.  The weight's columns col0 .. col0 + Nout
// are the piece; columns from `vocab` on do not exist for the softmax.
struct LossArgs : SplitArgs {
  int col0;
  int vocab;
  const int64_t* labels;
  int64_t ignore_index;
  const float* lse;     // LossGrad
  const float* dloss;   // LossDX
  float2* stats;        // LossStats: [2 n_tiles][M] (maximum, sum of exponentials) of 128 columns
  float* label_logit;   // LossStats: [M]
  float* acc;           // LossDX: fp32 [M][Nout] sums over the pieces
  int first, last;      // LossDX: no piece before / after this one
};

template <int kMode>
struct ModeTypes {
  struct Maps { CUtensorMap act, la, lb, out; };
  using Args = FusedArgs;
};
struct MapsPair { CUtensorMap act, la, lb, out, act2, la2, lb2; };
struct MapsGated : MapsPair { CUtensorMap g, u; };   // where kept (bf16, or codes of 8 bits)
struct MapsOne { CUtensorMap act, out; };            // out: P, dX; LossStats has none
template <> struct ModeTypes<kModeGatedFwd> { using Maps = MapsGated; using Args = GatedArgs; };
template <> struct ModeTypes<kModeGatedBwd> { using Maps = MapsPair; using Args = GatedArgs; };
template <> struct ModeTypes<kModeLossStats> { using Maps = MapsOne; using Args = LossArgs; };
template <> struct ModeTypes<kModeLossGrad> { using Maps = MapsOne; using Args = LossArgs; };
template <> struct ModeTypes<kModeLossDX> { using Maps = MapsOne; using Args = LossArgs; };

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

template <uint32_t kSel>
__device__ __forceinline__ uint32_t prmt_c(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "n"(kSel));
  return d;
}

// 8 packed nibbles (4 bytes, first weight in the high nibble of byte 0) ->
// 8 bf16 from the per-block table whose high and low bytes are split into
// H[0..3] and L[0..3] (entry j's byte in byte j%4 of H[j/4] / L[j/4]).  The
// byte permutes and logic share one pipe at half the issue rate, and its 21
// operations per 8 weights are what decoding costs.
__device__ __forceinline__ uint4 decode8(uint32_t p, const uint32_t (&H)[4],
                                         const uint32_t (&L)[4]) {
  // selector nibbles: low 3 bits pick a byte within a plane pair, bit 3
  // (moved to the "+4" position) picks the pair
  const uint32_t s = p & 0x77777777u;
  uint32_t b;
  // ((p >> 1) & 0x44444444) | 0x32103210 in one operation after the shift
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(b) : "r"(p >> 1), "r"(0x44444444u), "r"(0x32103210u));
  uint4 o;
  {
    const uint32_t hF = prmt(prmt(H[0], H[1], s), prmt(H[2], H[3], s), b);
    const uint32_t lF = prmt(prmt(L[0], L[1], s), prmt(L[2], L[3], s), b);
    o.x = prmt_c<0x4051u>(lF, hF);
    o.y = prmt_c<0x6273u>(lF, hF);
  }
  {
    const uint32_t s2 = s >> 16, b2 = b >> 16;
    const uint32_t hF = prmt(prmt(H[0], H[1], s2), prmt(H[2], H[3], s2), b2);
    const uint32_t lF = prmt(prmt(L[0], L[1], s2), prmt(L[2], L[3], s2), b2);
    o.z = prmt_c<0x4051u>(lF, hF);
    o.w = prmt_c<0x6273u>(lF, hF);
  }
  return o;
}

// Per-block table: entry j = bf16(C_j * a) (fp32 product, then bf16).
__device__ __forceinline__ void build_lut(const float* C, float a, uint32_t (&H)[4], uint32_t (&L)[4]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(C[2 * i] * a, C[2 * i + 1] * a);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    H[q] = prmt(w[2 * q], w[2 * q + 1], 0x7531u);
    L[q] = prmt(w[2 * q], w[2 * q + 1], 0x6420u);
  }
}

// The same for the NF4 codebook, its values immediates of the products.
__device__ __forceinline__ void build_lut_nf4(float a, uint32_t (&H)[4], uint32_t (&L)[4]) {
  constexpr float C[16] = {QNF4_TABLE_VALUES};
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(C[2 * i] * a, C[2 * i + 1] * a);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    H[q] = prmt(w[2 * q], w[2 * q + 1], 0x7531u);
    L[q] = prmt(w[2 * q], w[2 * q + 1], 0x6420u);
  }
}

// What one decoder thread needs for one K-step, loaded ahead of use.
struct RowFetch {
  uint4 p0, p1;   // 32 packed bytes of the row's NF4 block
  float sv;       // absmax, or the second-level scale (double quant)
  uint32_t q;     // scale code (double quant)
  bool valid;     // row inside the weight; false also for LoRA steps
  bool second;    // the gated backward's second weight
};

// Where a decoder thread loads next: K-step kk of work item `item`, and the NF4
// block that is its row of the decoded tile there.  Moves by additions; only at
// the end of an item (or of the gated backward's first weight, or of the
// contraction) does it look its block up again.
struct RowCursor {
  int item, kk;
  int until;      // K-steps of the item below which `blk` moves by `stride`
  bool valid;     // the row is inside the weight
  bool second;    // the gated backward's second weight
  int64_t blk, stride;
};

// Row R of the decoded tile of CTA `rank`.
template <int kMode>
__device__ __forceinline__ void seek_row(const typename ModeTypes<kMode>::Args& a, RowCursor& c, int R, int rank,
                                         int num_items, int nsteps) {
  c.valid = c.second = false;
  c.until = nsteps;
  c.blk = c.stride = 0;
  if (c.item >= num_items) return;
  int tile = c.item, kk = c.kk;
  if constexpr (mode_splits(kMode)) {
    const int tiles = a.m_tiles * a.n_tiles, split = tile / tiles;
    tile -= split * tiles;
    kk += split * a.steps;
    if (kk >= a.nk) return;
    if (a.nk - split * a.steps < nsteps) c.until = a.nk - split * a.steps;
    if (kMode == kModeGatedBwd) {
      const int half = a.nk / 2;
      if (kk >= half) {
        c.second = true;
        kk -= half;
      } else if (half - split * a.steps < c.until) {
        c.until = half - split * a.steps;
      }
    }
  }
  const int n0 = (tile / a.m_tiles) * mode_tile_cols(kMode);
  const int64_t bpr = a.Nw / 64;
  if constexpr (!mode_transposed(kMode)) {
    // columns of the tile: 128 per CTA, or the same 128 of each weight
    const int Rg = kMode == kModeGatedFwd ? R : kFBN * rank + R;
    int col = n0 + (Rg >> 6) * 64;
    if (col >= a.Nout) return;
    if constexpr (mode_loss(kMode)) col += a.col0;
    c.blk = (static_cast<int64_t>(kk) * 64 + (Rg & 63)) * bpr + col / 64;
    c.stride = 64 * bpr;
  } else {
    const int kw = n0 + kFBN * rank + R;
    if (kw >= a.Nout) return;
    if constexpr (mode_loss(kMode)) kk += a.col0 / 64;
    c.blk = kw * bpr + kk;
    c.stride = 1;
  }
  c.valid = true;
}

// `n` steps on; consecutive items of one pair are `stride` apart.
template <int kMode>
__device__ __forceinline__ void advance_row(const typename ModeTypes<kMode>::Args& a, RowCursor& c, int n, int R,
                                            int rank, int num_items, int nsteps, int stride) {
  c.kk += n;
  c.blk += n * c.stride;
  if (c.kk >= c.until) {
    while (c.kk >= nsteps) {
      c.kk -= nsteps;
      c.item += stride;
    }
    seek_row<kMode>(a, c, R, rank, num_items, nsteps);
  }
}

// The block at the cursor.
template <int kMode>
__device__ __forceinline__ void fetch_row(const typename ModeTypes<kMode>::Args& a, const RowCursor& c, int rank,
                                          RowFetch& f) {
  f.valid = c.valid;
  f.second = c.second;
  if (!c.valid) return;
  const uint8_t* packed = a.packed;
  const ScaleView* sv = &a.sv;
  if constexpr (mode_gated(kMode)) {
    if (kMode == kModeGatedFwd ? rank != 0 : c.second) {
      packed = a.packed2;
      sv = &a.sv2;
    }
  }
  const uint8_t* src = packed + c.blk * 32;
  // volatile asm: the loads issue here, K-steps before their use, instead of
  // being moved down to it
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(f.p0.x), "=r"(f.p0.y), "=r"(f.p0.z), "=r"(f.p0.w) : "l"(src));
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(f.p1.x), "=r"(f.p1.y), "=r"(f.p1.z), "=r"(f.p1.w) : "l"(src + 16));
  if (sv->code8 == nullptr) {
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(f.sv) : "l"(sv->absmax + c.blk));
  } else {
    // into a 32-bit register: a widening of a 16-bit one would wait for the load here
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(f.q) : "l"(sv->code8 + c.blk));
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(f.sv) : "l"(sv->s2 + (c.blk >> 8)));
  }
}

// Rows of a pair tile (the layer's own modes: always 512).
template <int kMode>
__device__ __forceinline__ int tile_rows(const typename ModeTypes<kMode>::Args& a) {
  if constexpr (kMode == kModeFwd || kMode == kModeBwd)
    return kFPairRows;
  else
    return a.rows;
}

// Whether the first of two LoRA steps goes before the last two K-steps: at the
// end the second one's tiles would be fetched only once the last K-step has left
// its stage.  (The gated forward of 1000 x 4096 x 11008: 149.5 us at the end, 147.5 so.)
template <int kMode>
__device__ __forceinline__ bool lora_early(int nsteps) { return mode_lora_steps(kMode) > 1 && nsteps >= 4; }

// Slices of 128 rows per CTA of the tile that starts at row m0 which hold rows
// of the activation (the layer's own modes always run both).
template <int kMode>
__device__ __forceinline__ int tile_slices(const typename ModeTypes<kMode>::Args& a, int m0) {
  if (kMode == kModeFwd || kMode == kModeBwd) return kFSlices;
  return tile_rows<kMode>(a) > 256 && a.M - m0 > 256 ? 2 : 1;
}

// 32 fp32 values as 32 bf16
__device__ __forceinline__ void pack_bf16x32(const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

// The ring a warp stores its rows through.  A lane holds a row of the
// accumulator, so its own stores would write 32 rows 16 bytes at a time, half a
// sector each; laid out in shared memory (64-byte swizzle: no bank conflict) a
// tile of 32 rows x 64 bytes leaves by one TMA store, which also drops the rows
// past M, while the warp goes on to the next.  (Measured at 4096 x 4096 x 11008:
// the gated forward that keeps g and u 606 us against 637 with direct stores, 578
// with eight warps instead of four; in 8 bits 607 against 742.)
struct RowStore {
  uint32_t base;   // shared address of the warp's slots, 1024-byte aligned
  uint32_t slot;
};

// One tile: this lane's 64 bytes of row `row0` + lane from element `x` on.  The
// whole warp takes part; row0 is below M.
__device__ __forceinline__ void store_rows(RowStore& rs, const CUtensorMap* map, int x, int row0, int lane,
                                           const uint32_t (&w)[16]) {
  if (lane == 0) bulk_wait_group_read<kFOutSlots - 1>();   // the slot's last tile has been read
  __syncwarp();
  const uint32_t at = rs.base + rs.slot * kFOutSlot;
  const uint32_t dst = at + lane * 64, sw = static_cast<uint32_t>((lane >> 1) & 3) << 4;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    sts128(dst + ((i << 4) ^ sw), make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, at, x, row0);
    bulk_commit_group();
  }
  rs.slot = (rs.slot + 1) % kFOutSlots;
}

// The same where a lane holds one column (x + lane) of the 32 rows, as the
// transposed modes' accumulators do: each row's 64 bytes are one store of the warp.
__device__ __forceinline__ void store_cols(RowStore& rs, const CUtensorMap* map, int x, int row0, int lane,
                                           const float (&v)[32]) {
  if (lane == 0) bulk_wait_group_read<kFOutSlots - 1>();
  __syncwarp();
  const uint32_t at = rs.base + rs.slot * kFOutSlot;
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k) {   // rows by the swizzle of their 16-byte chunks
    const uint32_t dst = at + ((static_cast<uint32_t>(lane >> 3) ^ k) << 4) + (lane & 7) * 2;
#pragma unroll
    for (uint32_t i = 2 * k; i < 32; i += 8) {
      const uint32_t p = pack_bf16x2(v[i], v[i + 1]);
      sts16(dst + i * 64, p);
      sts16(dst + i * 64 + 64, p >> 16);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, at, x, row0);
    bulk_commit_group();
  }
  rs.slot = (rs.slot + 1) % kFOutSlots;
}

__device__ __forceinline__ float round_bf16(float x) {
  return __uint_as_float(pack_bf16x2(x, 0.0f) << 16);
}

// The 8-bit codes of 64 accumulator columns rounded to bf16, exactly as
// qlora_act8_quantize would form them from the bf16 matrix (bf16 magnitudes order
// as integers, NaN and infinity above all finite values).
template <typename Release>
__device__ __forceinline__ void store_act8_block(RowStore& rs, const CUtensorMap* map, uint32_t taddr, int col,
                                                 int row0, int lane, bool in, float* scale, int32_t* d_status,
                                                 Release&& release) {
  uint32_t p[32];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t v[32];
    __syncwarp();
    tmem_ld_32x32b_x32(taddr + c * 32, v);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      p[16 * c + i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
      m = __vmaxu2(m, p[16 * c + i] & 0x7FFF7FFFu);
    }
  }
  release();
  const uint32_t top = max(m & 0xFFFFu, m >> 16);
  const float s = act8_scale(__uint_as_float(top << 16));
  const float inv = act8_inverse(s);
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x[8] = {p[8 * i],     p[8 * i + 1], p[8 * i + 2], p[8 * i + 3],
                           p[8 * i + 4], p[8 * i + 5], p[8 * i + 6], p[8 * i + 7]};
    const uint4 o = act8_codes16(x, s, inv);
    w[4 * i] = o.x;
    w[4 * i + 1] = o.y;
    w[4 * i + 2] = o.z;
    w[4 * i + 3] = o.w;
  }
  store_rows(rs, map, col, row0, lane, w);
  if (in) {
    *scale = s;
    if (top >= 0x7F80u) raise_status(d_status, QLORA_ERR_NONFINITE);
  }
}

// The epilogues call `release` once, when they have read the accumulator: the next
// tile's products go on while the last values are worked on and stored.

// Gated forward: 32 rows, one a lane, of 64 of the 128 g (columns 0 .. 127 of the
// accumulator) and 128 u (128 .. 255).
template <typename Release>
__device__ __forceinline__ void epilogue_gated(const GatedArgs& a, const MapsGated& maps, RowStore& rs,
                                               uint32_t tbase, int row0, int lane, int n0, int cols,
                                               Release&& release) {
  const int col0 = n0 + 64 * cols;
  if (row0 >= a.M || col0 >= a.Nout) {   // the same for the whole warp
    release();
    return;
  }
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int col = col0 + c * 32;
    __syncwarp();                       // the TMEM load takes the whole warp
    uint32_t vg[32], vu[32], w[16];
    tmem_ld_32x32b_x32(tbase + 64 * cols + c * 32, vg);
    tmem_ld_32x32b_x32(tbase + 128 + 64 * cols + c * 32, vu);
    tmem_ld_wait();
    if (c == 1 && a.keep != 2) release();
    if (a.keep == 1) {
      pack_bf16x32(vg, w);
      store_rows(rs, &maps.g, col, row0, lane, w);
      pack_bf16x32(vu, w);
      store_rows(rs, &maps.u, col, row0, lane, w);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i] = act_mul2(a.act, __uint_as_float(vg[2 * i]), __uint_as_float(vg[2 * i + 1]), __uint_as_float(vu[2 * i]),
                      __uint_as_float(vu[2 * i + 1]));
    store_rows(rs, &maps.out, col, row0, lane, w);
  }
  if (a.keep == 2) {
    const int64_t at = (row0 + lane) * static_cast<int64_t>(a.Nout / 64) + col0 / 64;
#pragma unroll 1
    for (int b = 0; b < 2; ++b)
      store_act8_block(rs, b == 0 ? &maps.g : &maps.u, tbase + 128 * b + 64 * cols, col0, row0, lane,
                       row0 + lane < a.M, (b == 0 ? a.Gs : a.Us) + at, a.d_status, [&] {
                         if (b == 1) release();
                       });
  }
}

// Loss statistics of this lane's row over 128 of the tile's columns: the running
// maximum m and the sum s of exp(l - m), and the label's logit where the
// label's column is here.
template <typename Release>
__device__ __forceinline__ void epilogue_loss_stats(const LossArgs& a, uint32_t tbase, int row, int n0, int cols,
                                                    Release&& release) {
  const bool in = row < a.M;
  const int64_t label = in ? a.labels[row] : -1;
  float m = -CUDART_INF_F, s = 0.0f;
  const int left = a.vocab - a.col0 - n0 - 128 * cols;   // columns of these that exist
  const int nc = left <= 0 ? 0 : (left < 128 ? (left + 31) / 32 : 4);
  if (nc == 0) release();
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    const int col = a.col0 + n0 + 128 * cols + c * 32;
    const int nv = left - c * 32;
    uint32_t v[32];
    __syncwarp();
    tmem_ld_32x32b_x32(tbase + 128 * cols + c * 32, v);
    tmem_ld_wait();
    if (c == nc - 1) release();
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < nv) top = fmaxf(top, __uint_as_float(v[i]));
    const float nm = fmaxf(m, top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < nv) sum += ex2((__uint_as_float(v[i]) - nm) * kLog2E);
    s = (m == nm ? s : s * ex2((m - nm) * kLog2E)) + sum;
    m = nm;
    const int64_t at = label - col;
    if (at >= 0 && at < 32 && at < nv) {
      float l = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i == static_cast<int>(at)) l = __uint_as_float(v[i]);
      a.label_logit[row] = l;
    }
  }
  if (in) a.stats[static_cast<int64_t>(n0 / kFAccCols * 2 + cols) * a.M + row] = make_float2(m, s);
}

// Whether a row's label counts.
__device__ __forceinline__ bool label_counts(const LossArgs& a, int row) {
  if (row >= a.M) return false;
  const int64_t label = a.labels[row];
  return label != a.ignore_index && label >= 0 && label < a.vocab;
}

// P = exp(l - lse) - onehot(label) of this lane's row, bf16; zero in the
// columns from `vocab` on and in rows whose label does not count.  dloss comes
// in behind the product with Ŵᵀ: in P it would be rounded with it, and alike in
// every row of a mean (-dloss at the label where the token was not expected).
template <typename Release>
__device__ __forceinline__ void epilogue_loss_grad(const LossArgs& a, const CUtensorMap* out, RowStore& rs,
                                                   uint32_t tbase, int row0, int lane, int n0, int cols,
                                                   Release&& release) {
  const int left = a.Nout - n0 - 128 * cols;   // columns of these, a multiple of 64
  const int nc = row0 >= a.M || left <= 0 ? 0 : (left < 128 ? 2 : 4);
  if (nc == 0) {
    release();
    return;
  }
  const int row = row0 + lane;
  const bool in = row < a.M;
  const int64_t label = in ? a.labels[row] : -1;
  const bool counts = label_counts(a, row);
  const float lse = in ? a.lse[row] : 0.0f;
  // once a row: a label that is neither ignored nor in the vocabulary
  if (a.col0 + n0 + cols == 0 && in && !counts && label != a.ignore_index)
    raise_status(a.d_status, QLORA_ERR_INVALID_ARG);
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    const int x = n0 + 128 * cols + c * 32;
    const int col = a.col0 + x;
    const int nv = a.vocab - col;
    const int64_t at = label - col;
    uint32_t v[32], w[16];
    __syncwarp();
    tmem_ld_32x32b_x32(tbase + 128 * cols + c * 32, v);
    tmem_ld_wait();
    if (c == nc - 1) release();
    float p[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float e = ex2((__uint_as_float(v[i]) - lse) * kLog2E);
      p[i] = counts && i < nv ? e - (i == at ? 1.0f : 0.0f) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
    store_rows(rs, out, x, row0, lane, w);
  }
}

// dX of one output column (x + lane) over 32 rows: times the row's dloss (0
// where the label does not count), added to the pieces before this one in fp32
// (without a result, so that no load waits between stores); the last piece
// adds the sums and rounds to bf16.  `scale` is dloss of row row0 + lane.
__device__ __forceinline__ void epilogue_loss_dx(const LossArgs& a, const CUtensorMap* out, RowStore& rs,
                                                 const uint32_t (&v)[32], float scale, int split, int x0, int lane,
                                                 int row0) {
  const int64_t ld = a.Nout;
  const int64_t at = row0 * ld + x0 + lane;
  const int nrows = x0 < a.Nout ? a.M - row0 : 0;   // (a multiple of 64: the same for the whole warp)
  if (nrows <= 0) return;
  float x[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]) * __shfl_sync(0xFFFFFFFFu, scale, i);
  if (a.splits > 1) {
    float* dst = a.part + static_cast<int64_t>(split) * a.M * ld + at;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < nrows) dst[i * ld] = x[i];
    return;
  }
  if (!a.last) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < nrows) {
        if (a.first)
          a.acc[at + i * ld] = x[i];
        else
          atomicAdd(a.acc + at + i * ld, x[i]);   // one thread per element: no order
      }
    return;
  }
  if (!a.first) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < nrows) x[i] += a.acc[at + i * ld];
  }
  store_cols(rs, out, x0, row0, lane, x);
}

// A split item's fp32 sums of one output column over 32 rows; false where the
// tile is not split.
__device__ __forceinline__ bool split_sums(const SplitArgs& a, const uint32_t (&v)[32], int split, int col,
                                           int row0) {
  if (a.splits <= 1) return false;
  if (col < a.Nout && row0 < a.M) {
    const int64_t ld = a.Nout;
    float* dst = a.part + (static_cast<int64_t>(split) * a.M + row0) * ld + col;
    const int nrows = a.M - row0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < nrows) dst[i * ld] = __uint_as_float(v[i]);
  }
  return true;
}
__device__ __forceinline__ bool split_sums(const FusedArgs&, const uint32_t (&)[32], int, int, int) { return false; }

// The split items' sums, in order, rounded to bf16 (four elements a thread).
__global__ void __launch_bounds__(256)
    split_join_kernel(const float4* __restrict__ part, int splits, int64_t quads, uint2* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < quads;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float4 s = part[i];
#pragma unroll 4
    for (int k = 1; k < splits; ++k) {
      const float4 v = part[k * quads + i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    out[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

template <int kMode>
__global__ void __launch_bounds__(kFThreads, 1)
    fused_nf4_gemm_kernel(const __grid_constant__ typename ModeTypes<kMode>::Maps maps,
                          const typename ModeTypes<kMode>::Args args) {
  constexpr bool kBwd = mode_transposed(kMode);
  constexpr int kLora = mode_lora_steps(kMode);
  constexpr int kTileCols = mode_tile_cols(kMode);
  constexpr bool kLayer = kMode == kModeFwd || kMode == kModeBwd;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kFAStages * kFA;
  uint8_t* sO = sB + kFBStages * kFB;   // the epilogue's staging
  float* t8 = reinterpret_cast<float*>(sO + kFOut);
  uint64_t* full_a = reinterpret_cast<uint64_t*>(t8 + 256);
  uint64_t* empty_a = full_a + kFAStages;
  uint64_t* full_b = empty_a + kFAStages;
  uint64_t* empty_b = full_b + kFBStages;
  uint64_t* tfull = empty_b + kFBStages;
  uint64_t* tempty = tfull + 1;   // [kFSlices]: one per accumulator
  uint64_t* drain = tempty + kFSlices;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  // (through a shuffle, so that the compiler knows it to be the same for the warp)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // the pair is the cluster (2 x 1 x 1): rank 0 issues the MMAs
  const int rank = static_cast<int>(blockIdx.x & 1);
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
  {
    bool dq = args.sv.code8 != nullptr;
    if constexpr (mode_gated(kMode)) dq = dq || args.sv2.code8 != nullptr;
    if (dq) build_t8(t8);
  }
  if (threadIdx.x == 0) {
    // Only CTA 0's full_a, full_b and tempty are waited on; every CTA's
    // empty_a, empty_b and tfull receive the pair MMA's multicast commits.
    for (int s = 0; s < kFAStages; ++s) {
      mbar_init(&full_a[s], 1);            // CTA 0's producer, plus both CTAs' bytes
      mbar_init(&empty_a[s], 1);
    }
    for (int s = 0; s < kFBStages; ++s) {
      mbar_init(&full_b[s], 2 * kFDecWarps);   // both CTAs' decoder warps
      mbar_init(&empty_b[s], 1);
    }
    mbar_init(tfull, 1);
    for (int h = 0; h < kFSlices; ++h) mbar_init(&tempty[h], 2 * kFEpiWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  // the peer's barriers are initialised before any arrival reaches them
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // work items: the tiles, or `splits` of each (item i: tile i % tiles)
  const int tiles = args.m_tiles * args.n_tiles;
  int num_tiles = tiles, nsteps = args.nk;
  if constexpr (mode_splits(kMode)) {
    num_tiles *= args.splits;
    nsteps = args.steps;
  }
  auto split_of = [&](int& item) -> int {
    if constexpr (mode_splits(kMode)) {
      const int s = item / tiles;
      item -= s * tiles;
      return s;
    }
    return 0;
  };
  pdl_launch_dependents();   // after this CTA holds its TMEM
  // the loss modes have no rank-r product before them: every input may come
  // from the kernel that precedes
  if constexpr (kLora == 0) pdl_wait();
  // Otherwise no wait for the preceding kernel here.  It is always this library's
  // rank-r product (Zc, or dZ), which lets this kernel launch only after all
  // kernels before it have completed: the activations, the weights and the
  // output buffer are final or free, and only the LoRA step's Zc (dZ) comes
  // from the preceding kernel; the producer waits before loading it.

  if (warp == 0) {
    // ------------------------------ TMA producer ---------------------------
    if (lane == 0) {
      tma_prefetch_desc(&maps.act);
      if constexpr (kLora > 0) {
        tma_prefetch_desc(&maps.la);
        tma_prefetch_desc(&maps.lb);
      }
      if constexpr (kLora > 1) {
        if constexpr (kBwd) tma_prefetch_desc(&maps.act2);
        tma_prefetch_desc(&maps.la2);
        tma_prefetch_desc(&maps.lb2);
      }
      uint32_t ia = 0;                          // activation-ring slot counter
      uint32_t last_parity[kFAStages];
#pragma unroll
      for (int s = 0; s < kFAStages; ++s) last_parity[s] = 2;
      bool ok = true;
      // take the next slot; CTA 0 arms its full barrier with both CTAs' bytes
      auto take = [&](uint32_t& s_out, uint32_t bytes) -> bool {
        const uint32_t s = ia % kFAStages, ph = (ia / kFAStages) & 1;
        if (*abort_flag || !mbar_wait(&empty_a[s], ph ^ 1)) return false;
        if (rank == 0) mbar_arrive_expect_tx(&full_a[s], 2 * bytes);
        last_parity[s] = ph;
        s_out = s;
        ++ia;
        return true;
      };
      auto bar0 = [&](uint32_t s) -> uint32_t { return mapa_shared(smem_u32(&full_a[s]), 0); };
      // the activation rows of slice h of this CTA
      auto act_row = [&](int m0, int h) -> int {
        return kMode == kModeFwd ? m0 + 256 * rank + 128 * h : m0 + 256 * h + 128 * rank;
      };
      bool lora_ready = false;
      for (int item = pair; item < num_tiles && ok; item += npairs) {
        int tile = item;
        const int split = split_of(tile);
        const int m0 = (tile % args.m_tiles) * tile_rows<kMode>(args);
        const int n0 = (tile / args.m_tiles) * kTileCols;
        const int nh = tile_slices<kMode>(args, m0);
        const uint32_t act_bytes = kLayer ? kFA : static_cast<uint32_t>(nh) * 16384u;
        // (steps past the contraction's end multiply zeros by zeros: boxes past
        // the end arrive as zero fill, and so do the decoders' rows)
        const int kk0 = split * nsteps;
        // LoRA step: Zc / dZ into one stage, B / A into the next
        auto lora = [&](int l) -> bool {
          if (kLora > 0 && !lora_ready) {
            pdl_wait();   // Zc (dZ) is the preceding kernel's output
            lora_ready = true;
          }
          const CUtensorMap *la = nullptr, *lb = nullptr;
          if constexpr (kLora > 0) { la = &maps.la; lb = &maps.lb; }
          if constexpr (kLora > 1) {
            if (l == 1) { la = &maps.la2; lb = &maps.lb2; }
          }
          uint32_t s1, s2;
          if (!take(s1, act_bytes)) return false;
          uint8_t* a = sA + s1 * kFA;
#pragma unroll
          for (int h = 0; h < kFSlices; ++h)
            if (h < nh) tma_load_2d_pair(a + h * 16384, la, bar0(s1), 0, act_row(m0, h));
          if (!take(s2, kFB)) return false;
          uint8_t* b = sA + s2 * kFA;
          if (!kBwd) {
            // B's columns of this CTA's half, two 64-column boxes (MN-major);
            // gated: the CTA's own B in its step, rows past the end (zeros) in the other's
            const int bx = kMode == kModeGatedFwd ? n0 : n0 + 128 * rank;
            const int by = kMode == kModeGatedFwd && l != rank ? 64 : 0;
#pragma unroll
            for (int nb = 0; nb < kFBN / 64; ++nb)
              tma_load_2d_pair(b + nb * 8192, lb, bar0(s2), bx + nb * 64, by);
          } else {
            // A's rows of this CTA's output columns (K-major)
            tma_load_2d_pair(b, lb, bar0(s2), 0, n0 + 128 * rank);
          }
          return true;
        };
        const bool early = lora_early<kMode>(nsteps) && split == 0;
        for (int kk = kk0; kk < kk0 + nsteps && ok; ++kk) {
          if (early && kk == nsteps - 2 && !lora(0)) { ok = false; break; }
          uint32_t s;
          if (!take(s, act_bytes)) { ok = false; break; }
          uint8_t* a = sA + s * kFA;
          const CUtensorMap* ma = &maps.act;
          int kx = kk * 64;
          if constexpr (kMode == kModeGatedBwd) {
            if (kk >= args.nk / 2) {
              ma = &maps.act2;
              kx -= args.nk / 2 * 64;
            }
          }
#pragma unroll
          for (int h = 0; h < kFSlices; ++h)
            if (h < nh) tma_load_2d_pair(a + h * 16384, ma, bar0(s), kx, act_row(m0, h));
        }
        if (!ok) break;
        if (split > 0) continue;
        for (int l = early ? 1 : 0; l < kLora && ok; ++l) ok = lora(l);
      }
      if (!ok) *abort_flag = 1;
      // CTA 0: let copies already in flight (its own and the peer's) land
      // before either CTA can exit
      if (rank == 0)
        for (int s = 0; s < kFAStages; ++s)
          if (last_parity[s] < 2) (void)mbar_wait(&full_a[s], last_parity[s]);
    }
  } else if (warp == 1) {
    // ------------------------- MMA issuer (CTA 0 only) ----------------------
    // The whole warp runs the loop and its elected lane issues: every
    // instruction of this warp waits for the decoders of its scheduler, so the
    // products' operands are kept to one addition each (descriptors differ from
    // the first stage's in their low word only).
    if (rank == 0) {
      // forward: D[m][n] += act[m][k] * Ŵtile[k][n] (tile MN-major, as B);
      // backward: D[n][m] += Ŵtile[n][k] * dY[m][k] (tile K-major, as A)
      constexpr uint32_t idesc = kBwd ? idesc_bf16_f32(256, kFAccCols, 0, 0)
                                      : idesc_bf16_f32(256, kFAccCols, 0, 1);
      // activation operand: slices 16 KB apart, 16-wide K slices 32 bytes apart;
      // weight operand: K slices 32 bytes (K-major) or 2 KB (MN-major) apart
      const uint64_t act0 = smem_desc(smem_u32(sA), 16, 1024);
      const uint64_t wgt0 = kBwd ? smem_desc(smem_u32(sB), 16, 1024) : smem_desc(smem_u32(sB), 8192, 1024);
      // the weight operand of a LoRA step lies in an activation stage
      const uint64_t lor0 = kBwd ? act0 : smem_desc(smem_u32(sA), 8192, 1024);
      constexpr uint32_t kWSlice = kBwd ? 2 : 128;
      const uint32_t acthi = static_cast<uint32_t>(act0 >> 32), wgthi = static_cast<uint32_t>(wgt0 >> 32);
      const uint32_t elected = elect_one();
      uint32_t sa = 0, pha = 0, sb = 0, phb = 0, tc = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_try_wait(bar, parity) || (!*abort_flag && mbar_wait(bar, parity));
      };
      auto next_a = [&]() {
        if (++sa == kFAStages) { sa = 0; pha ^= 1; }
      };
      // one 16-wide K slice of accumulator h: `al` the activation slice, `wl`
      // the weight slice (low words)
      auto mma = [&](int h, uint32_t al, uint32_t wl, uint32_t accum) {
        if (kBwd)
          umma_bf16_pair_lo(elected, tmem + h * kFAccCols, wl, wgthi, al + h * 1024, acthi, idesc, accum);
        else
          umma_bf16_pair_lo(elected, tmem + h * kFAccCols, al + h * 1024, acthi, wl, wgthi, idesc, accum);
      };
      for (int item = pair; item < num_tiles && ok; item += npairs, ++tc) {
        int tile = item;
        const int split = split_of(tile);
        const uint32_t tph = (tc & 1) ^ 1;       // parity of the previous tile's release
        const int nh = tile_slices<kMode>(args, (tile % args.m_tiles) * tile_rows<kMode>(args));
        auto lora = [&]() -> bool {
          const uint32_t s1 = sa;
          if (!wait(&full_a[s1], pha)) return false;
          next_a();
          const uint32_t s2 = sa;
          if (!wait(&full_a[s2], pha)) return false;
          next_a();
          tc_fence_after();
          const uint32_t al = static_cast<uint32_t>(act0) + s1 * (kFA >> 4);
          const uint32_t wl = static_cast<uint32_t>(lor0) + s2 * (kFA >> 4);
          for (int j = 0; j < args.rsteps; ++j)
#pragma unroll
            for (int h = 0; h < kFSlices; ++h)
              if (kLayer || h < nh) mma(h, al + j * 2, wl + j * kWSlice, 1u);
          umma_commit_pair_mc_if(elected, smem_u32(&empty_a[s1]), 0x3);
          umma_commit_pair_mc_if(elected, smem_u32(&empty_a[s2]), 0x3);
          return true;
        };
        const bool early = lora_early<kMode>(nsteps) && split == 0;
        for (int kk = 0; kk < nsteps; ++kk) {
          if (early && kk == nsteps - 2 && !lora()) { ok = false; break; }
          if (!wait(&full_a[sa], pha) || !wait(&full_b[sb], phb)) { ok = false; break; }
          tc_fence_after();
          const uint32_t al = static_cast<uint32_t>(act0) + sa * (kFA >> 4);
          const uint32_t wl = static_cast<uint32_t>(wgt0) + sb * (kFB >> 4);
          if (kk == 0) {
            // first K-step of a tile: each accumulator as soon as it is drained
#pragma unroll
            for (int h = 0; h < kFSlices; ++h) {
              if (!wait(&tempty[h], tph)) { ok = false; break; }
              tc_fence_after();
              if (kLayer || h < nh) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mma(h, al + j * 2, wl + j * kWSlice, j > 0 ? 1u : 0u);
              }
            }
            if (!ok) break;
          } else if (kLayer || nh == kFSlices) {
            // the two accumulators in turn: a product waits for the one before
            // it on the same accumulator (171 clocks from one to the next at N =
            // 256, 128 where two alternate)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int h = 0; h < kFSlices; ++h) mma(h, al + j * 2, wl + j * kWSlice, 1u);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) mma(0, al + j * 2, wl + j * kWSlice, 1u);
          }
          umma_commit_pair_mc_if(elected, smem_u32(&empty_a[sa]), 0x3);
          umma_commit_pair_mc_if(elected, smem_u32(&empty_b[sb]), 0x3);
          next_a();
          if (++sb == kFBStages) { sb = 0; phb ^= 1; }
        }
        if (!ok) break;
        for (int l = early ? 1 : 0; l < kLora && split == 0 && ok; ++l) ok = lora();
        if (!ok) break;
        umma_commit_pair_mc_if(elected, smem_u32(tfull), 0x3);
      }
      if (!ok) *abort_flag = 1;
      umma_commit_pair_mc_if(elected, smem_u32(drain), 0x1);
      (void)mbar_wait(drain, 0);
    }
  } else if (warp < 2 + kFDecAll) {
    // ------------------------------ decoders -------------------------------
    const int grp = (warp - 2) / kFDecWarps;   // this warp's turn among the groups
    const int R = threadIdx.x - 64 - grp * kFBN;   // row of this CTA's decoded tile
    // this CTA's weight (the gated forward's CTA 1 has the second one)
    const ScaleView* sv1 = &args.sv;
    if constexpr (kMode == kModeGatedFwd) {
      if (rank != 0) sv1 = &args.sv2;
    }
    const float off1 = sv1->code8 != nullptr ? __ldg(sv1->offset) : 0.0f;
    float off2 = 0.0f;
    if constexpr (kMode == kModeGatedBwd) {
      if (args.sv2.code8 != nullptr) off2 = __ldg(args.sv2.offset);
    }
    bool ok = true;
    // steps still to come for this pair, and this group's among them
    int64_t left = pair < num_tiles ? static_cast<int64_t>((num_tiles - pair + npairs - 1) / npairs) * nsteps - grp : 0;
    RowCursor at{};                            // the step being loaded
    at.item = pair + grp / nsteps * npairs;
    at.kk = grp % nsteps;
    seek_row<kMode>(args, at, R, rank, num_tiles, nsteps);
    uint32_t ib = static_cast<uint32_t>(grp);
    // One K-step: wait for a free weight stage, decode this thread's row.
    auto step = [&](const RowFetch& f) {
      const uint32_t s = ib % kFBStages, ph = (ib / kFBStages) & 1;
      if (!mbar_try_wait(&empty_b[s], ph ^ 1) && (*abort_flag || !mbar_wait(&empty_b[s], ph ^ 1))) {
        ok = false;
        return;
      }
      // row R of the stage, its 16-byte chunk bits holding the swizzle
      const uint32_t brow = smem_u32(sB) + s * kFB + R * 128 + ((R & 7) << 4);
      if (f.valid) {
        const ScaleView* sv = sv1;
        float off = off1;
        if constexpr (kMode == kModeGatedBwd) {
          if (f.second) { sv = &args.sv2; off = off2; }
        }
        const float a = sv->code8 == nullptr
                            ? f.sv
                            : __fadd_rn(__fmul_rn(t8[f.q], f.sv), off);
        uint32_t H[4], L[4];
        build_lut(kNF4g + 16 * sv->codebook, a, H, L);
        const uint32_t pw[8] = {f.p0.x, f.p0.y, f.p0.z, f.p0.w, f.p1.x, f.p1.y, f.p1.z, f.p1.w};
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) sts128(brow ^ (c << 4), decode8(pw[c], H, L));
      } else {
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) sts128(brow ^ (c << 4), make_uint4(0, 0, 0, 0));
      }
      // the rows are visible to the tensor core (async proxy), then CTA 0's
      // barrier of the stage counts this warp
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&full_b[s]), 0));
      left -= kFDecGroups;
      ib += kFDecGroups;
    };
    // Three prefetch slots consumed and refilled in place (no register moves
    // that would wait on loads still in flight).
    RowFetch q0{}, q1{}, q2{};
    auto fetch = [&](RowFetch& f) {
      fetch_row<kMode>(args, at, rank, f);
      advance_row<kMode>(args, at, kFDecGroups, R, rank, num_tiles, nsteps, npairs);
    };
    fetch(q0);
    fetch(q1);
    fetch(q2);
    while (ok && left > 0) {
      step(q0);
      fetch(q0);
      if (!ok || left <= 0) break;
      step(q1);
      fetch(q1);
      if (!ok || left <= 0) break;
      step(q2);
      fetch(q2);
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ------------------------------ epilogue -------------------------------
    const int q = warp & 3;
    uint32_t tc = 0;
    bool ok = true;
    const int ew = warp - (2 + kFDecAll), cols = ew >> 2;   // which half of an accumulator's columns
    RowStore rs{smem_u32(sO) + static_cast<uint32_t>(ew * kFOutSlots * kFOutSlot), 0};
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);   // CTA 0's release barriers
    for (int item = pair; item < num_tiles && ok; item += npairs, ++tc) {
      int tile = item;
      const int split = split_of(tile);
      const int m0 = (tile % args.m_tiles) * tile_rows<kMode>(args);
      const int n0 = (tile / args.m_tiles) * kTileCols;
      const int nh = tile_slices<kMode>(args, m0);
      // loss: dloss of the lane's row in the next 32 (0 where its label does not
      // count), loaded 32 rows ahead
      auto row_scale = [&](int row) -> float {
        if constexpr (kMode == kModeLossDX) {
          if (label_counts(args, row)) return args.dloss[row];
        }
        return 0.0f;
      };
      float next_scale = row_scale(m0 + 128 * cols + lane);
      if (*abort_flag || !mbar_wait(tfull, tc & 1)) { ok = false; break; }
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < kFSlices; ++h) {
        const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * kFAccCols;
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty0 + static_cast<uint32_t>(h) * 8u);
        };
        if (!kLayer && h >= nh) {
          release();
          continue;
        }
        // rows of the forward layouts: the layer's slices lie 128 apart
        const int row0 = kMode == kModeFwd ? m0 + 256 * rank + 128 * h + q * 32 : m0 + 256 * h + 128 * rank + q * 32;
        if constexpr (kMode == kModeGatedFwd) {
          epilogue_gated(args, maps, rs, tbase, row0, lane, n0, cols, release);
        } else if constexpr (kMode == kModeLossStats) {
          epilogue_loss_stats(args, tbase, row0 + lane, n0, cols, release);
        } else if constexpr (kMode == kModeLossGrad) {
          epilogue_loss_grad(args, &maps.out, rs, tbase, row0, lane, n0, cols, release);
        } else if constexpr (kMode == kModeFwd) {
          const int left = args.Nout - n0 - 128 * cols;   // columns of these, a multiple of 64
          const int nc = row0 >= args.M || left <= 0 ? 0 : (left < 128 ? 2 : 4);
          if (nc == 0) release();
#pragma unroll 1
          for (int c = 0; c < nc; ++c) {
            uint32_t v[32], w[16];
            __syncwarp();
            tmem_ld_32x32b_x32(tbase + 128 * cols + c * 32, v);
            tmem_ld_wait();
            if (c == nc - 1) release();
            pack_bf16x32(v, w);
            store_rows(rs, &maps.out, n0 + 128 * cols + c * 32, row0, lane, w);
          }
        } else {
#pragma unroll 1
          for (int c = 4 * cols; c < 4 * cols + 4; ++c) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld_32x32b_x32(tbase + c * 32, v);
            tmem_ld_wait();
            if (c == 4 * cols + 3) release();
            // lane = output column x0 + lane, 32 consecutive output rows
            const int x0 = n0 + 128 * rank + q * 32, y0 = m0 + h * kFAccCols + c * 32;
            if constexpr (kMode == kModeLossDX) {
              const float scale = next_scale;
              next_scale = row_scale((c < 4 * cols + 3 ? y0 + 32 : y0 - 96 + kFAccCols) + lane);
              epilogue_loss_dx(args, &maps.out, rs, v, scale, split, x0, lane, y0);
            } else if (kMode == kModeGatedBwd && split_sums(args, v, split, x0 + lane, y0)) {
            } else if (x0 < args.Nout && y0 < args.M) {
              float x[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]);
              store_cols(rs, &maps.out, x0, y0, lane, x);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();   // the staged rows have left
    if (!ok) *abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the pair MMA, the peer's copies or the peer's
  // arrivals may still reach it
  cluster_sync_all();
  if (*abort_flag && threadIdx.x == 0) raise_status(args.d_status, QLORA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Items a dX tile is cut into: as many as keep every pair of the sizing SM
// count busy, of at least kSplitSteps K-steps each (an item's start and its
// sums cost about as much as four steps).
// (4 and 16 measured within 1 % of 8 on the loss and the gated block at 200 to 333 rows.)
constexpr int kSplitSteps = 8;
constexpr int kSizingPairs = 74;   // whatever the device, so that results depend on the shape only
inline int dx_most_splits(int tiles, int nk) {
  const int s = kSizingPairs / tiles, m = nk / kSplitSteps;
  const int most = s < m ? s : m;
  return most < 2 ? 1 : most;
}
inline int dx_splits(int tiles, int nk) {
  const int s = dx_most_splits(tiles, nk);   // equal items may need fewer
  const int steps = (nk + s - 1) / s;
  return (nk + steps - 1) / steps;
}

// Workspace of a split dX (M x cols), 0 when it is not split.  Grows with nk, so
// that a size asked for with more K-steps serves fewer.
inline size_t split_bytes(int64_t M, int64_t cols, int64_t nk) {
  const int64_t tiles = ((M + kFPairRows - 1) / kFPairRows) * ((cols + kFPairCols - 1) / kFPairCols);
  if (tiles > kSizingPairs) return 0;
  const int s = dx_most_splits(static_cast<int>(tiles), static_cast<int>(nk));
  return s > 1 ? (static_cast<size_t>(s) * M * cols * 4 + 255) / 256 * 256 : 0;
}

// Rows of the tiles of a forward layout (n_tiles column tiles): 256 where all of
// those run at once.  A tile of 256 rows takes about 0.9 of the time of one of
// 512 (its weights' decode is the same), so more waves of them cost more.
inline void set_rows(SplitArgs& a) {
  a.rows = (a.M + 255) / 256 * a.n_tiles <= kSizingPairs ? 256 : 512;
  a.m_tiles = (a.M + a.rows - 1) / a.rows;
}

// Fills the split of a dX launch; `part` from split_bytes (null: not split).
inline void set_split(SplitArgs& a, float* part) {
  a.rows = kFPairRows;
  const int tiles = a.m_tiles * a.n_tiles;
  a.splits = part != nullptr ? dx_splits(tiles, a.nk) : 1;
  a.steps = (a.nk + a.splits - 1) / a.splits;
  a.part = part;
}

inline cudaError_t launch_split_join(const SplitArgs& a, uint16_t* out, int prof_kind, cudaStream_t st) {
  const int64_t quads = static_cast<int64_t>(a.M) * a.Nout / 4;
  const int64_t want = (quads + 255) / 256;
  cudaError_t e;
  {
    ProfScope prof(prof_kind, st);
    e = launch_pdl(split_join_kernel, dim3(static_cast<unsigned>(want < 1184 ? want : 1184)), dim3(256), 0, st, 1,
                   reinterpret_cast<const float4*>(a.part), a.splits, quads, reinterpret_cast<uint2*>(out));
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int kMode>
cudaError_t set_fused_attr() {
  static DeviceOnce once;
  return once.run([](int) {
    return cudaFuncSetAttribute(fused_nf4_gemm_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kFSmem));
  });
}

}  // namespace
}  // namespace qnf4
