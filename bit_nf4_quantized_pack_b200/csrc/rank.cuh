// Rank-r contractions on sm_100a (X·A, G·Bᵀ, Xᵀ·dZ, Gᵀ·Zc) and their host-side
// launchers, shared by the layer (linear.cu) and the operators built on it:
//   skinny_gemm_kernel  split-K over a thread-block cluster, alone on the GPU
//   rank_rows_kernel    one CTA per row tile, on the SMs a fused GEMM leaves free
// Every translation unit that includes this file gets its own copy of what it
// uses.
#pragma once

#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "tmap.cuh"

namespace qnf4 {
namespace {

// ===========================================================================
// Skinny contraction:  D[m'][n'] = sum_k' A(m',k') * B(n',k'),  n' < 64.
// A tiles are 128 x 64 and B tiles 64 x 64 (bf16), each either K-major
// (rows of 64 contiguous k') or MN-major (rows of 64 contiguous m'/n'), all
// with the 128-byte swizzle.  blockIdx.x = 128-row tile, blockIdx.y = split.
// ===========================================================================
constexpr int kSkW = 2;                  // 64-wide k' boxes per stage
constexpr int kSkStages = 8 / kSkW;
constexpr int kSkA = 16384 * kSkW, kSkB = 8192 * kSkW;
constexpr int kSkThreads = 192;  // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr size_t kSkSmem = 1024 + kSkStages * (kSkA + kSkB) + 256;
static_assert(kSkStages * 8 * 3 + 16 <= 256, "skinny barriers and flags fit the tail");

struct SkinnyArgs {
  int Mp;            // rows of D
  int nk;            // number of k' blocks (64 * kSkW wide)
  int kb_per_split;  // k' blocks per split
  int splits;        // = cluster size along y (<= 8)
  int ncols;         // columns of D that are summed (the rank, or the padded rank)
  int nout;          // columns written to `out` (<= ncols)
  float scale;
  int mode;          // 0: bf16 out[Mp][ld]; 1: fp32 out[Mp][ld]; 2: fp32 out[nout][Mp];
                     // 3: bf16 out[nout][Mp]
  void* out;
  int ld;
  uint16_t* out2;    // mode 0 only, may be null: all ncols columns again, bf16 [Mp][ld2]
  int ld2;
  int32_t* d_status;
};

// A second contraction of the same shape in the same launch (blockIdx.z = 1):
// its own operands and outputs.
struct SkinnySecond {
  void* out;
  uint16_t* out2;
};

// The A operand as an 8-bit activation checkpoint (rows k', columns m'), read
// as X̂ᵀ: codes [rows][cols], scales [rows][cols / 64].
struct SkinnyA8 {
  const int8_t* codes;
  const float* scales;
  int rows, cols;
};

template <bool kPair, bool kA8>
struct SkinnyMaps {
  CUtensorMap a, b;
};
template <>
struct SkinnyMaps<true, false> {
  CUtensorMap a, b, a2, b2;
};
template <>
struct SkinnyMaps<false, true> {
  CUtensorMap b;
};
template <>
struct SkinnyMaps<true, true> {
  CUtensorMap b, b2;
};

constexpr int kSkA8Group = 4 * kSkW;   // decoder warps of a stage of the 8-bit A operand
constexpr int kSkA8Turns = 2;          // groups of them that take stages in turn
constexpr int kSkA8Warps = kSkA8Group * kSkA8Turns;
constexpr int kSkA8Ahead = 2;          // of its stages, whose codes a decoder thread has in flight

constexpr int kSkRedLd = 65;   // fp32 words per row of the split-sum buffer (bank spread)
constexpr int kSkMaxSplits = 8;  // portable cluster size

// One of the 256 decoder threads of an MN-major 8-bit A operand's stage.  Eight
// warps share its 256 rows (two boxes of two 64-column halves of 64 k' rows): warp w
// has box w >> 2, half (w >> 1) & 1 and 32 rows of it, a thread 16 codes of four
// rows eight apart, so that four lanes read a row's 64 bytes together (a lane
// to a row costs the L1 four times as many passes) and a store phase's eight
// lanes meet all banks.
struct A8Decoder {
  const SkinnyA8& a8;
  int box, hh, kr, c, col;
  int64_t bpr;

  struct Rows {
    uint4 p[4];
    float s[4];
  };

  __device__ __forceinline__ A8Decoder(const SkinnyA8& a, int t, int m0)
      : a8(a), box(t >> 7), hh((t >> 6) & 1), kr(((t >> 5) & 1) * 32 + ((t & 31) >> 2)), c(t & 3),
        col(m0 + ((t >> 6) & 1) * 64), bpr(a.cols / 64) {}

  // the codes of k' block kb (zeros from block `end` on and past the matrix)
  __device__ __forceinline__ void fetch(Rows& r, int kb, int end) const {
    const int row = (kb * kSkW + box) * 64 + kr;
    const int left = kb < end && col < a8.cols ? a8.rows - row : 0;   // rows from this one on
    const int8_t* p = a8.codes + static_cast<int64_t>(row) * a8.cols + col + 16 * c;
    const float* sp = a8.scales + row * bpr + col / 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.s[i] = 0.0f;
      r.p[i] = make_uint4(0, 0, 0, 0);
      if (8 * i < left) {
        // volatile asm: the loads issue here, stages before their use
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.p[i].x), "=r"(r.p[i].y), "=r"(r.p[i].z), "=r"(r.p[i].w)
                     : "l"(p));
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(r.s[i]) : "l"(sp));
      }
      p += 8 * static_cast<int64_t>(a8.cols);
      sp += 8 * bpr;
    }
  }

  // their values into the stage, in the 128-byte swizzle of a box
  __device__ __forceinline__ void store(const Rows& r, uint8_t* stage) const {
    const uint32_t rowp = smem_u32(stage) + box * 16384 + hh * 8192 + kr * 128;
    const uint32_t sw = static_cast<uint32_t>(kr & 7) << 4;   // kr + 8 i: the same swizzle
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t q[4] = {r.p[i].x, r.p[i].y, r.p[i].z, r.p[i].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[4];
        act8_values4(q[j], r.s[i], v);
        o[2 * j] = pack_bf16x2(v[0], v[1]);
        o[2 * j + 1] = pack_bf16x2(v[2], v[3]);
      }
      const uint32_t at = rowp + i * 1024;
      sts128(at + ((c << 5) ^ sw), make_uint4(o[0], o[1], o[2], o[3]));
      sts128(at + (((c << 5) | 16) ^ sw), make_uint4(o[4], o[5], o[6], o[7]));
    }
  }

  // This turn's K blocks of kb0 .. kb1 - 1.
  template <typename Wait>
  __device__ __forceinline__ bool run(int kb0, int kb1, int turn, uint8_t* sA, uint64_t* full, int lane,
                                      Wait&& wait_empty) const {
    Rows r[kSkA8Ahead];
    const int first = kb0 + turn;
#pragma unroll
    for (int i = 0; i < kSkA8Ahead; ++i) fetch(r[i], first + i * kSkA8Turns, kb1);
    for (int kb = first; kb < kb1; kb += kSkA8Ahead * kSkA8Turns) {
#pragma unroll
      for (int i = 0; i < kSkA8Ahead; ++i) {
        const int k = kb + i * kSkA8Turns;
        if (k < kb1) {
          const int g = k - kb0, s = g % kSkStages;
          if (!wait_empty(g)) return false;
          store(r[i], sA + s * kSkA);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          fetch(r[i], k + kSkA8Ahead * kSkA8Turns, kb1);
        }
      }
    }
    return true;
  }
};

// kA8: A is an MN-major 8-bit checkpoint.  Sixteen more warps (after the
// epilogue's) decode it instead of TMA: a tile row is 64 codes of one k' row
// and one scale, written as 64 bf16 in the 128-byte swizzle that the box would
// have; two groups of eight take stages in turn (one alone spent 2.2 thousand
// clocks a stage, 40 % of them issuing) and load four stages ahead.
template <bool kAmn, bool kBmn, bool kPair = false, bool kA8 = false>
__global__ void __launch_bounds__(kSkThreads + (kA8 ? kSkA8Warps * 32 : 0), 1)
    skinny_gemm_kernel(const __grid_constant__ SkinnyMaps<kPair, kA8> maps, SkinnyArgs args,
                       SkinnySecond second, SkinnyA8 a8) {
  static_assert(!kA8 || kAmn, "an 8-bit operand is read transposed");
  const CUtensorMap* pA = nullptr;
  const CUtensorMap* pB = &maps.b;
  if constexpr (!kA8) pA = &maps.a;
  if constexpr (kPair) {
    if (blockIdx.z != 0) {
      if constexpr (!kA8) pA = &maps.a2;
      pB = &maps.b2;
      args.out = second.out;
      args.out2 = second.out2;
    }
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kSkStages * kSkA;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + kSkStages * kSkB);
  uint64_t* empty = full + kSkStages;
  uint64_t* done = empty + kSkStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
  float* red = reinterpret_cast<float*>(sA);   // [128][kSkRedLd], after the last MMA

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = blockIdx.x * 128;
  const int kb0 = blockIdx.y * args.kb_per_split;
  const int kb1 = min(args.nk, kb0 + args.kb_per_split);
  const int nkb = kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSkStages; ++s) {
      mbar_init(&full[s], kA8 ? 1 + kSkA8Group : 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // Wait for the preceding kernel first and only then let the next one
  // launch: the fused kernel that follows a rank-r product then knows that
  // every kernel before this one has completed, and reads its activations
  // and weights at once, waiting only for this kernel's result.
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0 && lane == 0) {
    if constexpr (!kA8) tma_prefetch_desc(pA);
    tma_prefetch_desc(pB);
    for (int i = 0; i < nkb; ++i) {
      const int s = i % kSkStages;
      const uint32_t ph = (i / kSkStages) & 1;
      if (!mbar_wait(&empty[s], ph ^ 1)) { *abort_flag = 1; break; }
      const int kb = kb0 + i;
      mbar_arrive_expect_tx(&full[s], kA8 ? kSkB : kSkA + kSkB);
#pragma unroll
      for (int w = 0; w < kSkW; ++w) {
        const int kx = (kb * kSkW + w) * 64;   // boxes past the end arrive as zero fill
        uint8_t* a = sA + s * kSkA + w * 16384;
        uint8_t* b = sB + s * kSkB + w * 8192;
        if constexpr (!kA8) {
          if (kAmn) {
            tma_load_2d(a, pA, &full[s], m0, kx);
            tma_load_2d(a + 8192, pA, &full[s], m0 + 64, kx);
          } else {
            tma_load_2d(a, pA, &full[s], kx, m0);
          }
        }
        if (kBmn)
          tma_load_2d(b, pB, &full[s], 0, kx);
        else
          tma_load_2d(b, pB, &full[s], kx, 0);
      }
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 64, kAmn ? 1 : 0, kBmn ? 1 : 0);
    bool ok = true;
    for (int i = 0; i < nkb; ++i) {
      const int s = i % kSkStages;
      const uint32_t ph = (i / kSkStages) & 1;
      if (!mbar_wait(&full[s], ph)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < kSkW; ++w) {
        const uint32_t a0 = smem_u32(sA + s * kSkA + w * 16384), b0 = smem_u32(sB + s * kSkB + w * 8192);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t ad = kAmn ? smem_desc(a0 + j * 2048, 8192, 1024) : smem_desc(a0 + j * 32, 16, 1024);
          const uint64_t bd = kBmn ? smem_desc(b0 + j * 2048, 8192, 1024) : smem_desc(b0 + j * 32, 16, 1024);
          umma_bf16(tmem, ad, bd, idesc, (i > 0 || w > 0 || j > 0) ? 1u : 0u);
        }
      }
      umma_commit(&empty[s]);
    }
    if (!ok) *abort_flag = 1;
    umma_commit(done);  // also drains whatever was issued
  } else if (kA8 && warp >= 6) {
    // decoders of the 8-bit operand
    const int t = threadIdx.x - kSkThreads;
    const A8Decoder d(a8, t % (kSkA8Group * 32), m0);
    if (!d.run(kb0, kb1, t / (kSkA8Group * 32), sA, full, lane,
               [&](int u) { return mbar_wait(&empty[u % kSkStages], ((u / kSkStages) & 1) ^ 1); }))
      *abort_flag = 1;
  } else if (warp >= 2) {
    // Epilogue, part 1: this split's fp32 sums into shared memory (the A ring
    // is free once the last MMA has completed).
    const int q = warp & 3;
    const bool okd = mbar_wait(done, 0);
    tc_fence_after();
    if (!okd) *abort_flag = 1;
    const int row = q * 32 + lane;
    const int nc = args.ncols;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (c * 32 < nc) {
        uint32_t v[32];
        if (okd) {
          tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 32, v);
          tmem_ld_wait();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c * 32 + i < nc) red[row * kSkRedLd + c * 32 + i] = okd ? __uint_as_float(v[i]) : 0.0f;
      }
    }
  }
  // Part 2: the splits of a row tile are one thread-block cluster along y.
  // Each adds a share of the tile's rows over all splits, in split order,
  // reading the others' sums from distributed shared memory, and writes out.
  cluster_sync_all();
  if (warp >= 2 && warp < 6) {
    const int S = args.splits;
    const int rank = static_cast<int>(blockIdx.y);   // cluster spans all of y
    const int rows_per = (128 + S - 1) / S;
    const int r0 = rank * rows_per;
    const int nrow = min(rows_per, 128 - r0);
    const int nc = args.ncols;
    const int total = nrow > 0 ? nrow * nc : 0;
    const uint32_t red_s = smem_u32(red);
    for (int e = threadIdx.x - 64; e < total; e += 128) {
      // modes 2 and 3 write columns of out: let consecutive threads take consecutive rows
      const int rr = args.mode >= 2 ? e % nrow : e / nc;
      const int cc = args.mode >= 2 ? e / nrow : e % nc;
      const int lrow = r0 + rr, grow = m0 + lrow;
      // all S loads in flight first, then the sum in split order
      const uint32_t off = red_s + static_cast<uint32_t>((lrow * kSkRedLd + cc) * 4);
      float part[kSkMaxSplits];
#pragma unroll
      for (int sp = 0; sp < kSkMaxSplits; ++sp)
        part[sp] = sp < S ? ld_dsmem_f32(off, static_cast<uint32_t>(sp)) : 0.0f;
      float acc = 0.0f;
#pragma unroll
      for (int sp = 0; sp < kSkMaxSplits; ++sp)
        if (sp < S) acc += part[sp];
      acc *= args.scale;
      if (grow < args.Mp) {
        if (args.mode == 0) {
          const uint16_t v = static_cast<uint16_t>(pack_bf16x2(acc, 0.0f) & 0xFFFFu);
          if (cc < args.nout) static_cast<uint16_t*>(args.out)[static_cast<int64_t>(grow) * args.ld + cc] = v;
          if (args.out2 != nullptr) args.out2[static_cast<int64_t>(grow) * args.ld2 + cc] = v;
        } else if (cc < args.nout) {
          if (args.mode == 1)
            static_cast<float*>(args.out)[static_cast<int64_t>(grow) * args.ld + cc] = acc;
          else if (args.mode == 3)
            static_cast<uint16_t*>(args.out)[static_cast<int64_t>(cc) * args.Mp + grow] =
                static_cast<uint16_t>(pack_bf16x2(acc, 0.0f) & 0xFFFFu);
          else
            static_cast<float*>(args.out)[static_cast<int64_t>(cc) * args.Mp + grow] = acc;
        }
      }
    }
  }
  cluster_sync_all();   // no CTA leaves while another still reads its sums
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) raise_status(args.d_status, QLORA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}


// ===========================================================================
// Rank-r product on a few SMs beside the fused GEMM:  D = scale * A B (the
// operand layouts and output modes of the split kernel above), the whole
// contraction per 128-row tile in one CTA (no split), tiles blockIdx.x,
// + gridDim.x, ...  The fused GEMM leaves these SMs free (its grid is sized
// to the fewest pairs that need no more waves of tiles): Zc (dZ) here lets
// it start at once and wait for the product only at its LoRA step, and dA,
// dB here run beside dX.  Same roles as above: warp 0 TMA, warp 1 MMA into
// one TMEM accumulator (128 x 64 fp32), warps 2..5 read it (released on
// `tempty` per tile), scale and store.  kPair: the tiles of a second product of
// the same sizes follow those of the first.
// ===========================================================================
template <bool kAmn, bool kBmn, bool kPair>
__global__ void __launch_bounds__(kSkThreads, 1)
    rank_rows_kernel(const __grid_constant__ SkinnyMaps<kPair, false> maps, SkinnyArgs args, SkinnySecond other) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kSkStages * kSkA;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + kSkStages * kSkB);
  uint64_t* empty = full + kSkStages;
  uint64_t* done = empty + kSkStages;
  uint64_t* tempty = done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tempty + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tiles = (args.Mp + 127) / 128, tiles = kPair ? 2 * m_tiles : m_tiles;
  const int nkb = args.nk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSkStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(tempty, 4);   // the four epilogue warps
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // wait for the preceding kernel, then let the fused GEMM launch
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
    int g = 0;   // stage uses over all tiles
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const CUtensorMap *pA = &maps.a, *pB = &maps.b;
      int m0 = t * 128;
      if constexpr (kPair) {
        if (t >= m_tiles) {
          pA = &maps.a2;
          pB = &maps.b2;
          m0 -= m_tiles * 128;
        }
      }
      for (int i = 0; i < nkb; ++i, ++g) {
        const int s = g % kSkStages;
        const uint32_t ph = (g / kSkStages) & 1;
        if (g >= kSkStages && !mbar_wait(&empty[s], ph ^ 1)) { ok = false; break; }
        mbar_arrive_expect_tx(&full[s], kSkA + kSkB);
#pragma unroll
        for (int w = 0; w < kSkW; ++w) {
          const int kx = (i * kSkW + w) * 64;   // boxes past the end arrive as zero fill
          uint8_t* a = sA + s * kSkA + w * 16384;
          uint8_t* b = sB + s * kSkB + w * 8192;
          if (kAmn) {
            tma_load_2d(a, pA, &full[s], m0, kx);
            tma_load_2d(a + 8192, pA, &full[s], m0 + 64, kx);
          } else {
            tma_load_2d(a, pA, &full[s], kx, m0);
          }
          if (kBmn)
            tma_load_2d(b, pB, &full[s], 0, kx);
          else
            tma_load_2d(b, pB, &full[s], kx, 0);
        }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, 64, kAmn ? 1 : 0, kBmn ? 1 : 0);
    int g = 0, it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++it) {
      // the epilogue has read the previous tile's accumulator
      if (it > 0 && !mbar_wait(tempty, (it - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      for (int i = 0; i < nkb; ++i, ++g) {
        const int s = g % kSkStages;
        const uint32_t ph = (g / kSkStages) & 1;
        if (!mbar_wait(&full[s], ph)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int w = 0; w < kSkW; ++w) {
          const uint32_t a0 = smem_u32(sA + s * kSkA + w * 16384), b0 = smem_u32(sB + s * kSkB + w * 8192);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t ad = kAmn ? smem_desc(a0 + j * 2048, 8192, 1024) : smem_desc(a0 + j * 32, 16, 1024);
            const uint64_t bd = kBmn ? smem_desc(b0 + j * 2048, 8192, 1024) : smem_desc(b0 + j * 32, 16, 1024);
            umma_bf16(tmem, ad, bd, idesc, (i > 0 || w > 0 || j > 0) ? 1u : 0u);
          }
        }
        umma_commit(&empty[s]);
      }
      umma_commit(done);   // one phase per tile (also drains an aborted tile)
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 2) {
    const int q = warp & 3;   // TMEM lanes 32q .. 32q + 31
    const int nc = args.ncols;
    int it = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
      const bool okd = mbar_wait(done, it & 1);
      tc_fence_after();
      if (!okd) { *abort_flag = 1; break; }
      const bool second = kPair && t >= m_tiles;
      void* const out = second ? other.out : args.out;
      uint16_t* const out2 = second ? other.out2 : args.out2;
      const int grow = (second ? t - m_tiles : t) * 128 + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (c * 32 < nc) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 32, v);
          tmem_ld_wait();
          if (grow < args.Mp && args.mode == 0) {
            uint16_t* o = static_cast<uint16_t*>(out) + static_cast<int64_t>(grow) * args.ld;
            uint16_t* o2 = out2 != nullptr ? out2 + static_cast<int64_t>(grow) * args.ld2 : nullptr;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int cc = c * 32 + i;
              if (cc < nc) {
                // (0 + v) * scale: the split kernel's sum and rounding for one split
                const uint16_t b = static_cast<uint16_t>(
                    pack_bf16x2((0.0f + __uint_as_float(v[i])) * args.scale, 0.0f) & 0xFFFFu);
                if (cc < args.nout) o[cc] = b;
                if (o2 != nullptr) o2[cc] = b;
              }
            }
          } else if (grow < args.Mp) {
            // fp32: mode 1 out[Mp][ld], mode 2 out[nout][Mp] (consecutive lanes,
            // consecutive rows); mode 3: bf16 out[nout][Mp]
            float* o = static_cast<float*>(out);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int cc = c * 32 + i;
              if (cc < args.nout) {
                const float x = (0.0f + __uint_as_float(v[i])) * args.scale;
                if (args.mode == 1)
                  o[static_cast<int64_t>(grow) * args.ld + cc] = x;
                else if (args.mode == 3)
                  static_cast<uint16_t*>(out)[static_cast<int64_t>(cc) * args.Mp + grow] =
                      static_cast<uint16_t>(pack_bf16x2(x, 0.0f) & 0xFFFFu);
                else
                  o[static_cast<int64_t>(cc) * args.Mp + grow] = x;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) raise_status(args.d_status, QLORA_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

// Zero-padded copy of a rows x r bf16 matrix into rows x rp (rp = r rounded
// up to a multiple of 8), so that every row starts on a 16-byte boundary as
// the tensor maps need.  Only used when r is not a multiple of 8.
__global__ void __launch_bounds__(256) pad_cols_kernel(const uint16_t* __restrict__ src,
                                                       int64_t rows, int r,
                                                       uint16_t* __restrict__ dst, int rp) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = rows * rp;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / rp;
    const int col = static_cast<int>(i - row * rp);
    dst[i] = col < r ? src[row * r + col] : static_cast<uint16_t>(0);
  }
}
// ===========================================================================
// Host side
// ===========================================================================

// K splits of a rank-r contraction: one CTA per SM (the kernel's shared
// memory allows no second), so the grid is kept to a single wave.
// The SM count that fixes split counts and the rank-r path, whatever the
// device: results (the fp32 summation order of the rank-r products) depend on
// the shape only.
constexpr int g_ws_sms = 148;

int skinny_splits(int Mp, int nk, int num_sms) {
  const int mt = (Mp + 127) / 128;
  int want = num_sms / mt;
  if (want > kSkMaxSplits) want = kSkMaxSplits;
  if (want < 1) want = 1;
  if (want > nk) want = nk;
  const int per = (nk + want - 1) / want;
  return (nk + per - 1) / per;
}

struct WsCursor {
  char* p;
  size_t left;
  bool ok = true;
  void* take(size_t bytes) {
    bytes = (bytes + 255) & ~static_cast<size_t>(255);
    if (bytes > left) { ok = false; return nullptr; }
    void* r = p;
    p += bytes;
    left -= bytes;
    return r;
  }
};

size_t align256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

template <bool A, bool B, bool kPair, bool kA8>
cudaError_t set_skinny_attr() {
  static DeviceOnce once;
  return once.run([](int) {
    return cudaFuncSetAttribute(skinny_gemm_kernel<A, B, kPair, kA8>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSkSmem));
  });
}

template <bool A, bool B, bool kPair, bool kA8>
cudaError_t launch_skinny(const SkinnyMaps<kPair, kA8>& maps, SkinnyArgs a, int Kp, int splits,
                          SkinnySecond second, SkinnyA8 a8, cudaStream_t st) {
  cudaError_t e = set_skinny_attr<A, B, kPair, kA8>();
  if (e != cudaSuccess) return e;
  a.nk = (Kp + 64 * kSkW - 1) / (64 * kSkW);
  a.kb_per_split = (a.nk + splits - 1) / splits;
  a.splits = (a.nk + a.kb_per_split - 1) / a.kb_per_split;
  {
    ProfScope prof(kProfSkinny, st);
    e = launch_pdl(skinny_gemm_kernel<A, B, kPair, kA8>, dim3((a.Mp + 127) / 128, a.splits, kPair ? 2 : 1),
                   dim3(kSkThreads + (kA8 ? kSkA8Warps * 32 : 0), 1, 1), kSkSmem, st, a.splits, maps, a,
                   second, a8);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// D = scale * A(m',k') B(n',k'): one launch, split-K sums added in-kernel.
// ncols columns of D are summed; the first nout go to `out`, and in mode 0 all
// ncols also go to out2 (a padded copy) when it is not null.
template <bool kAmn, bool kBmn>
cudaError_t run_skinny(const CUtensorMap& ta, const CUtensorMap& tb, int Mp, int Kp, int ncols,
                       float scale, int mode, void* out, int ld, int splits, int32_t* d_status,
                       cudaStream_t st, int nout = -1, uint16_t* out2 = nullptr, int ld2 = 0) {
  SkinnyArgs a{};
  a.Mp = Mp;
  a.ncols = ncols;
  a.nout = nout < 0 ? ncols : nout;
  a.scale = scale;
  a.mode = mode;
  a.out = out;
  a.ld = ld;
  a.out2 = out2;
  a.ld2 = ld2;
  a.d_status = d_status;
  return launch_skinny<kAmn, kBmn, false, false>(SkinnyMaps<false, false>{ta, tb}, a, Kp, splits,
                                                 SkinnySecond{}, SkinnyA8{}, st);
}

template <bool A, bool B, bool kPair>
cudaError_t set_rank_rows_attr() {
  static DeviceOnce once;
  return once.run([](int) {
    return cudaFuncSetAttribute(rank_rows_kernel<A, B, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSkSmem));
  });
}

// Pairs of the fused GEMM: the fewest that keep its number of waves of tiles
// (so the SMs it leaves free cost it nothing).
int fused_pairs(int tiles, int sms) {
  const int most = sms / 2 > 0 ? sms / 2 : 1;
  const int waves = (tiles + most - 1) / most;
  const int pairs = waves > 0 ? (tiles + waves - 1) / waves : 1;
  return pairs < 1 ? 1 : pairs;
}

// CTAs for rank-r products streaming `bytes` beside the fused GEMM of `tiles`
// pair tiles, or 0 for the split kernel.  Decided for the sizing SM count
// (not the device's), so the forward and the backward's recompute make the
// same choice and form Zc alike: the SMs the fused GEMM leaves free (an even
// number), when there are at least 8 of them and each streams at most
// mb_per_sm MB (done long before the fused GEMM needs the product).
int rank_rows_ctas(double bytes, int tiles, double mb_per_sm) {
  const int free_sms = g_ws_sms - 2 * fused_pairs(tiles, g_ws_sms);
  if (free_sms < 8) return 0;
  if (bytes > mb_per_sm * 1e6 * free_sms) return 0;
  return free_sms;
}

template <bool kAmn, bool kBmn, bool kPair>
cudaError_t launch_rank_rows(const SkinnyMaps<kPair, false>& maps, SkinnyArgs a, int Kp, int ctas,
                             SkinnySecond second, cudaStream_t st) {
  cudaError_t e = set_rank_rows_attr<kAmn, kBmn, kPair>();
  if (e != cudaSuccess) return e;
  // at most one CTA per tile, in pairs (a 2 x 1 cluster, so that the SMs left
  // to the fused GEMM's pairs stay in pairs)
  const int tiles = (a.Mp + 127) / 128 * (kPair ? 2 : 1);
  if (ctas > tiles) ctas = tiles;
  ctas = (ctas + 1) & ~1;
  a.nk = (Kp + 64 * kSkW - 1) / (64 * kSkW);
  a.kb_per_split = a.nk;
  a.splits = 1;
  {
    ProfScope prof(kProfSkinny, st);
    e = launch_pdl_pair(rank_rows_kernel<kAmn, kBmn, kPair>, dim3(static_cast<unsigned>(ctas)),
                        dim3(kSkThreads, 1, 1), kSkSmem, st, maps, a, second);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// D = scale * A(m',k') B(n',k') by rank_rows_kernel on `ctas` CTAs; modes as
// for run_skinny (0: bf16 out, and all ncols columns again into out2 when it
// is not null; 1: fp32 out[Mp][ld]; 2: fp32 out[nout][Mp]).
template <bool kAmn, bool kBmn>
cudaError_t run_rank_rows(const CUtensorMap& ta, const CUtensorMap& tb, int Mp, int Kp, int ncols,
                          float scale, int mode, void* out, int ld, int ctas, int32_t* d_status,
                          cudaStream_t st, int nout = -1, uint16_t* out2 = nullptr, int ld2 = 0) {
  SkinnyArgs a{};
  a.Mp = Mp;
  a.ncols = ncols;
  a.nout = nout < 0 ? ncols : nout;
  a.scale = scale;
  a.mode = mode;
  a.out = out;
  a.ld = ld;
  a.out2 = out2;
  a.ld2 = ld2;
  a.d_status = d_status;
  return launch_rank_rows<kAmn, kBmn, false>(SkinnyMaps<false, false>{ta, tb}, a, Kp, ctas, SkinnySecond{}, st);
}

constexpr CUtensorMapDataType kBF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
constexpr CUtensorMapSwizzle kSW128 = CU_TENSOR_MAP_SWIZZLE_128B;
constexpr CUtensorMapSwizzle kSW64 = CU_TENSOR_MAP_SWIZZLE_64B;

int rsteps_of(int r) { return (r + 15) / 16; }

// Rank rounded up to a multiple of 8: the row pitch (rp * 2 bytes) of every
// rank-r operand read by TMA must be a multiple of 16 bytes.
int padded_rank(int r) { return (r + 7) & ~7; }

cudaError_t launch_pad(const uint16_t* src, int64_t rows, int r, uint16_t* dst, int rp,
                       cudaStream_t st) {
  const int64_t want = (rows * rp + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want < 592 ? want : 592);
  cudaError_t e;
  {
    ProfScope prof(kProfOther, st);
    e = launch_pdl(pad_cols_kernel, dim3(grid), dim3(256), 0, st, 1, src, rows, r, dst, rp);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// The same for several matrices of one rank in one launch (blockIdx.y).
struct PadSet {
  const uint16_t* src[4];
  uint16_t* dst[4];
  int64_t rows[4];
};

__global__ void __launch_bounds__(256) pad_sets_kernel(PadSet p, int r, int rp) {
  pdl_launch_dependents();
  pdl_wait();
  const int m = blockIdx.y;
  const int64_t total = p.rows[m] * rp;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / rp;
    const int col = static_cast<int>(i - row * rp);
    p.dst[m][i] = col < r ? p.src[m][row * r + col] : static_cast<uint16_t>(0);
  }
}

inline cudaError_t launch_pad_sets(const PadSet& p, int n, int r, int rp, cudaStream_t st) {
  int64_t most = 1;
  for (int i = 0; i < n; ++i) most = p.rows[i] > most ? p.rows[i] : most;
  const int64_t want = (most * rp + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want < 296 ? want : 296);
  cudaError_t e;
  {
    ProfScope prof(kProfOther, st);
    e = launch_pdl(pad_sets_kernel, dim3(grid, static_cast<unsigned>(n)), dim3(256), 0, st, 1, p, r, rp);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace
}  // namespace qnf4
