// Forward and backward of the NF4 frozen-base LoRA linear layer on sm_100a.
//
// Page "QLoRA：冻结的 4-bit 权重怎样参与一次微调":
//   §量化基座与可训练支路怎样相加      Z = X·A,  Y = X·Ŵ + c·Z·B
//   §冻结权重为什么仍然需要输入梯度    dZ = c·G·Bᵀ, dX = G·Ŵᵀ + dZ·Aᵀ,
//                                     dA = Xᵀ·dZ,  dB = c·Zᵀ·G
//
// Kernels launched from here:
//   skinny_gemm_kernel   (rank.cuh) rank-r contractions (X·A, G·Bᵀ, Xᵀ·dZ, Gᵀ·Zc): TMA
//                        for both operands (or a decoded 8-bit X), tcgen05 MMA
//                        with N = 64, split-K over the CTAs of a cluster, each of
//                        which adds a share of the rows over all of them through
//                        distributed shared memory.
//   rank_rows_kernel     (rank.cuh) the same unsplit, on the SMs that the fused GEMM
//                        leaves free.
//   fused_nf4_gemm_kernel  (fused.cuh) Y = X·Ŵ + Zc·B (forward) and dX = G·Ŵᵀ + dZ·Aᵀ
//                        (backward): persistent CTA pairs, warp-specialised; TMA
//                        brings activation tiles, decoder warps load packed
//                        nibbles from global memory and turn them into bf16
//                        operand tiles in shared memory, a converged warp's
//                        elected lane issues tcgen05.mma into TMEM, and the
//                        rank-r LoRA term is one extra K-step of the same
//                        accumulator.
// The M <= 16 forward (a GEMV) is in gemv.cu.
#include <atomic>
#include <cfloat>
#include <mutex>

#include "common.cuh"
#include "fused.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "rank.cuh"
#include "tmap.cuh"

namespace qnf4 {


// A library-owned stream per device for work that runs beside the caller's
// stream, and the two events of one fork and join.  Created on first use
// (retried after a failure, e.g. inside a stream capture that forbids it);
// g_side_mu is held from a fork to its join, so concurrent callers never
// interleave their records and waits on the shared events.
struct SideStream {
  cudaStream_t s = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};
static std::mutex g_side_mu;
static SideStream g_side[64];

static SideStream* side_stream() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  SideStream& ss = g_side[dev];
  if (ss.s == nullptr) {
    int least = 0, greatest = 0;
    cudaDeviceGetStreamPriorityRange(&least, &greatest);
    cudaStream_t s = nullptr;
    cudaEvent_t f = nullptr, j = nullptr;
    if (cudaStreamCreateWithPriority(&s, cudaStreamNonBlocking, least) != cudaSuccess ||
        cudaEventCreateWithFlags(&f, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&j, cudaEventDisableTiming) != cudaSuccess) {
      if (s != nullptr) cudaStreamDestroy(s);
      if (f != nullptr) cudaEventDestroy(f);
      (void)cudaGetLastError();
      return nullptr;
    }
    ss.fork = f;
    ss.join = j;
    ss.s = s;
  }
  return &ss;
}

// Whether work on `side` may depend on work on `st`: `side` is in no capture, or in
// the one that `st` is in.  (Only a fork takes it into one, under g_side_mu.)
static bool may_fork(cudaStream_t st, cudaStream_t side) {
  cudaStreamCaptureStatus a, b;
  unsigned long long ida = 0, idb = 0;
  if (cudaStreamGetCaptureInfo(st, &a, &ida) != cudaSuccess ||
      cudaStreamGetCaptureInfo(side, &b, &idb) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  return b == cudaStreamCaptureStatusNone ||
         (b == cudaStreamCaptureStatusActive && a == cudaStreamCaptureStatusActive && ida == idb);
}

SideFork::SideFork(cudaStream_t st, bool wanted) : lock_(g_side_mu), st_(st), side_(st) {
  SideStream* ss = wanted ? side_stream() : nullptr;
  if (ss != nullptr && may_fork(st, ss->s)) {
    if (cudaEventRecord(ss->fork, st) == cudaSuccess)
      ss_ = ss;
    else
      (void)cudaGetLastError();
  }
  if (ss_ == nullptr) lock_.unlock();
}

cudaStream_t SideFork::enter() {
  if (ss_ != nullptr) {
    if (cudaStreamWaitEvent(ss_->s, ss_->fork, 0) == cudaSuccess) {
      side_ = ss_->s;
    } else {
      (void)cudaGetLastError();   // in order; what else is wrong shows in the launches
      ss_ = nullptr;
    }
  }
  return side_;
}

cudaError_t SideFork::join() {
  if (ss_ == nullptr) return cudaSuccess;
  const cudaError_t e = cudaEventRecord(ss_->join, side_);
  return e == cudaSuccess ? cudaStreamWaitEvent(st_, ss_->join, 0) : e;
}

size_t linear_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r) {
  const int rp = padded_rank(r);
  // A zero-padded to rp columns when r is not a multiple of 8
  const size_t apad = rp != r ? align256(static_cast<size_t>(K) * rp * 2) : 0;
  if (M > 16) {
    // the rank-r kernel adds its splits in shared memory; a padded copy of Zc
    // for the fused kernel's TMA when r is not a multiple of 8
    return rp != r ? apad + align256(static_cast<size_t>(M) * rp * 2) : 0;
  }
  return apad;   // the GEMV adds its K splits inside a thread-block cluster
}

size_t linear_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r) {
  (void)N;
  const int rp = padded_rank(r);
  // dZ, and Zc when the caller recomputes it instead of saving it (or a padded
  // copy of the caller's Zc), both bf16 M x rp; A padded to rp columns
  return 2 * align256(static_cast<size_t>(M) * rp * 2) +
         (rp != r ? align256(static_cast<size_t>(K) * rp * 2) : 0);
}

cudaError_t launch_linear_fwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                              const uint8_t* packed, ScaleView sv, const uint16_t* A,
                              const uint16_t* B, float c, uint16_t* Y, uint16_t* Zc, void* ws,
                              size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms) {
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  const int rp = padded_rank(r);
  const bool pad = rp != r;
  cudaError_t e = cudaSuccess;
  // A zero-padded to rp columns (16-byte row pitch for TMA) when r % 8 != 0
  const uint16_t* At = A;
  if (pad) {
    uint16_t* Ap = static_cast<uint16_t*>(cur.take(static_cast<size_t>(K) * rp * 2));
    if (!cur.ok) return cudaErrorInvalidValue;
    e = launch_pad(A, K, r, Ap, rp, st);
    if (e != cudaSuccess) return e;
    At = Ap;
  }
  if (!cur.ok) return cudaErrorInvalidValue;
  // Zc = bf16(c * X A): A operand X (K-major), B operand A (MN-major over r)
  CUtensorMap tX, tAl, tZc, tBl, tY;
  if (!make_tmap_2d(&tX, X, kBF16, 2, M, K, K, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tAl, At, kBF16, 2, K, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (M <= 16) {
    // one launch: weights streamed once, X·A and its split sums in the same
    // cluster, Zc and Y written (the GEMV's own SM count fixes its splits)
    return launch_gemv(M, K, N, r, X, packed, sv, At, rp, B, c, Y, Zc, r, false, d_status, st,
                       num_sms);
  }

  // rank-r product for the tensor-core path: Zc = bf16(c * X A), and a copy
  // padded to rp columns for the fused kernel's TMA when r % 8 != 0
  uint16_t* Zp = nullptr;
  if (pad) {
    Zp = static_cast<uint16_t*>(cur.take(static_cast<size_t>(M) * rp * 2));
    if (!cur.ok) return cudaErrorInvalidValue;
  }
  {
    // beside the fused GEMM on the SMs it leaves free, or split-K before it
    const int fwd_tiles = static_cast<int>(((M + kFPairRows - 1) / kFPairRows) *
                                           ((N + kFPairCols - 1) / kFPairCols));
    const int rows_ctas = rank_rows_ctas(2.0 * M * K, fwd_tiles, 2.5);
    if (rows_ctas > 0) {
      e = run_rank_rows<false, true>(tX, tAl, static_cast<int>(M), static_cast<int>(K), rp, c, 0, Zc,
                                     r, rows_ctas, d_status, st, r, Zp, rp);
    } else {
      const int Sz = skinny_splits(static_cast<int>(M), static_cast<int>(K / 64), g_ws_sms);
      e = run_skinny<false, true>(tX, tAl, static_cast<int>(M), static_cast<int>(K), rp, c, 0, Zc, r,
                                  Sz, d_status, st, r, Zp, rp);
    }
    if (e != cudaSuccess) return e;
  }
  e = set_fused_attr<kModeFwd>();
  if (e != cudaSuccess) return e;
  if (!make_tmap_2d(&tZc, pad ? Zp : Zc, kBF16, 2, M, rp, rp, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tBl, B, kBF16, 2, r, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tY, Y, kBF16, 2, M, N, N, 32, 32, kSW64)) return cudaErrorInvalidValue;
  FusedArgs fa;
  fa.M = static_cast<int>(M);
  fa.Nout = static_cast<int>(N);
  fa.Nw = static_cast<int>(N);
  fa.nk = static_cast<int>(K / 64);
  fa.rsteps = rsteps_of(r);
  fa.m_tiles = static_cast<int>((M + kFPairRows - 1) / kFPairRows);   // pair tiles of 512 rows
  fa.n_tiles = static_cast<int>((N + kFPairCols - 1) / kFPairCols);   // and 256 columns
  fa.sv = sv;
  fa.packed = packed;
  fa.d_status = d_status;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // persistent pairs of CTAs (a cluster of 2 x 1): the fewest pairs that
  // keep the number of waves of tiles
  const int grid = fused_pairs(fa.m_tiles * fa.n_tiles, sms);
  {
    ProfScope prof(kProfFusedFwd, st);
    e = launch_pdl_pair(fused_nf4_gemm_kernel<kModeFwd>, dim3(2 * grid), dim3(kFThreads), kFSmem,
                        st, ModeTypes<kModeFwd>::Maps{tX, tZc, tBl, tY}, fa);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_linear_bwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* dY,
                              const uint16_t* X, const uint16_t* Zc, const uint8_t* packed,
                              ScaleView sv, const uint16_t* A, const uint16_t* B, float c,
                              uint16_t* dX, void* dA, void* dB, void* ws, size_t ws_bytes,
                              int32_t* d_status, cudaStream_t st, int num_sms, bool grad_bf16,
                              const int8_t* X8, const float* X8_scales) {
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  const int rp = padded_rank(r);
  const bool pad = rp != r;
  // dZ and the working copy of Zc are bf16 M x rp (row pitch 16-byte aligned)
  uint16_t* dZ = static_cast<uint16_t*>(cur.take(static_cast<size_t>(M) * rp * 2));
  uint16_t* Zc_ws = static_cast<uint16_t*>(cur.take(static_cast<size_t>(M) * rp * 2));
  uint16_t* Ap = pad ? static_cast<uint16_t*>(cur.take(static_cast<size_t>(K) * rp * 2)) : nullptr;
  const int Sz = skinny_splits(static_cast<int>(M), static_cast<int>(N / 64), g_ws_sms);
  const int nkm = static_cast<int>((M + 63) / 64);
  const int Sa = skinny_splits(static_cast<int>(K), nkm, g_ws_sms);
  const int Sb = skinny_splits(static_cast<int>(N), nkm, g_ws_sms);
  if (!cur.ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  const uint16_t* At = A;
  if (pad) {
    e = launch_pad(A, K, r, Ap, rp, st);
    if (e != cudaSuccess) return e;
    At = Ap;
  }
  if (Zc == nullptr && M <= 16) {
    // saved-activation policy "recompute": Zc = bf16(c X A) exactly as the
    // forward forms it for M <= 16 (the GEMV kernel, its splits and sums)
    e = launch_gemv(M, K, N, r, X, packed, sv, At, rp, B, c, nullptr, Zc_ws, rp, true, d_status, st,
                    num_sms);
    if (e != cudaSuccess) return e;
    Zc = Zc_ws;
  } else if (Zc == nullptr) {
    // saved-activation policy "recompute": Zc = bf16(c X A) exactly as the
    // forward forms it (same kernel, same splits, so the same bits)
    CUtensorMap tXf, tAf;
    if (!make_tmap_2d(&tXf, X, kBF16, 2, M, K, K, 64, 128, kSW128)) return cudaErrorInvalidValue;
    if (!make_tmap_2d(&tAf, At, kBF16, 2, K, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
    // the forward's choice of kernel and split, so the same bits
    const int fwd_tiles = static_cast<int>(((M + kFPairRows - 1) / kFPairRows) *
                                           ((N + kFPairCols - 1) / kFPairCols));
    const int rows_ctas = rank_rows_ctas(2.0 * M * K, fwd_tiles, 2.5);
    if (rows_ctas > 0) {
      e = run_rank_rows<false, true>(tXf, tAf, static_cast<int>(M), static_cast<int>(K), rp, c, 0,
                                     Zc_ws, rp, rows_ctas, d_status, st);
    } else {
      const int Sf = skinny_splits(static_cast<int>(M), static_cast<int>(K / 64), g_ws_sms);
      e = run_skinny<false, true>(tXf, tAf, static_cast<int>(M), static_cast<int>(K), rp, c, 0, Zc_ws,
                                  rp, Sf, d_status, st);
    }
    if (e != cudaSuccess) return e;
    Zc = Zc_ws;
  } else if (pad) {
    e = launch_pad(Zc, M, r, Zc_ws, rp, st);
    if (e != cudaSuccess) return e;
    Zc = Zc_ws;
  }

  CUtensorMap tG, tBk, tXmn, tdZ, tGmn, tZcmn, tAl;
  // dZ = c * G B^T : A operand G (K-major over N), B operand B (K-major: rows r, cols N);
  // B's rows past r arrive as zero fill, so dZ's padding columns are zero
  if (!make_tmap_2d(&tG, dY, kBF16, 2, M, N, N, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tBk, B, kBF16, 2, r, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  {
    const int dx_tiles = static_cast<int>(((M + kFPairRows - 1) / kFPairRows) *
                                          ((K + kFPairCols - 1) / kFPairCols));
    const int rows_ctas = rank_rows_ctas(2.0 * M * N, dx_tiles, 2.5);
    if (rows_ctas > 0)
      e = run_rank_rows<false, false>(tG, tBk, static_cast<int>(M), static_cast<int>(N), rp, c, 0, dZ,
                                      rp, rows_ctas, d_status, st);
    else
      e = run_skinny<false, false>(tG, tBk, static_cast<int>(M), static_cast<int>(N), rp, c, 0, dZ, rp,
                                   Sz, d_status, st);
  }
  if (e != cudaSuccess) return e;
  // dA = X^T dZ : A operand X^T (MN-major over K), B operand dZ (MN-major over r)
  if (X8 == nullptr && !make_tmap_2d(&tXmn, X, kBF16, 2, M, K, K, 64, 64, kSW128)) return cudaErrorInvalidValue;
  // (columns of dZ past rp arrive as TMA zero fill)
  if (!make_tmap_2d(&tdZ, dZ, kBF16, 2, M, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  // dB^T = G^T Zc : A operand G^T (MN-major over N), B operand Zc (MN-major over r)
  if (!make_tmap_2d(&tGmn, dY, kBF16, 2, M, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tZcmn, Zc, kBF16, 2, M, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  // dX = G W^T + dZ A^T
  e = set_fused_attr<kModeBwd>();
  if (e != cudaSuccess) return e;
  if (!make_tmap_2d(&tAl, At, kBF16, 2, K, rp, rp, 64, kFBN, kSW128)) return cudaErrorInvalidValue;
  CUtensorMap tdZa;
  if (!make_tmap_2d(&tdZa, dZ, kBF16, 2, M, rp, rp, 64, 128, kSW128)) return cudaErrorInvalidValue;
  CUtensorMap tdX;
  if (!make_tmap_2d(&tdX, dX, kBF16, 2, M, K, K, 32, 32, kSW64)) return cudaErrorInvalidValue;
  FusedArgs fa;
  fa.M = static_cast<int>(M);
  fa.Nout = static_cast<int>(K);
  fa.Nw = static_cast<int>(N);
  fa.nk = static_cast<int>(N / 64);
  fa.rsteps = rsteps_of(r);
  fa.m_tiles = static_cast<int>((M + kFPairRows - 1) / kFPairRows);   // pair tiles of 512 dY rows
  fa.n_tiles = static_cast<int>((K + kFPairCols - 1) / kFPairCols);   // and 256 output columns
  fa.sv = sv;
  fa.packed = packed;
  fa.d_status = d_status;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // persistent pairs of CTAs (a cluster of 2 x 1): the fewest pairs that
  // keep the number of waves of tiles
  const int grid = fused_pairs(fa.m_tiles * fa.n_tiles, sms);

  // dX on the caller's stream first; dA and dB, which need only dZ, Zc, X and
  // G, on the side stream after dZ, so their CTAs take the SMs that dX's
  // partial last wave of tiles leaves idle.  The caller's stream then waits
  // for them: to the caller the call is ordered as one operation on st.
  // (in order for the smaller backwards of an 8-bit input or with bf16 gradients)
  const bool in_order = (X8 != nullptr || grad_bf16) && !worth_forking(M, K, N);
  SideFork fork(st, !prof_timing(kProfSkinny) && !in_order);
  {
    ProfScope prof(kProfFusedBwd, st);
    e = launch_pdl_pair(fused_nf4_gemm_kernel<kModeBwd>, dim3(2 * grid), dim3(kFThreads), kFSmem, st,
                        ModeTypes<kModeBwd>::Maps{tG, tdZa, tAl, tdX}, fa);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  const cudaStream_t s2 = fork.enter();
  // dA, dB on the SMs dX leaves free when they can stream their 2 x M x
  // (K + N) bytes there well within dX, else split-K
  const int dx_tiles = fa.m_tiles * fa.n_tiles;
  const int dadb_ctas = rank_rows_ctas(2.0 * M * (K + N), dx_tiles, 5.0);
  const int modeA = grad_bf16 ? 0 : 1, modeB = grad_bf16 ? 3 : 2;
  auto run_db = [&]() {
    return dadb_ctas > 0
               ? run_rank_rows<true, true>(tGmn, tZcmn, static_cast<int>(N), static_cast<int>(M), r, 1.0f,
                                           modeB, dB, r, dadb_ctas, d_status, s2)
               : run_skinny<true, true>(tGmn, tZcmn, static_cast<int>(N), static_cast<int>(M), r, 1.0f, modeB,
                                        dB, r, Sb, d_status, s2);
  };
  if (X8 != nullptr) {
    // an 8-bit X: dB first, then dA with its decode, split over all SMs that dX
    // has left by then (on the free SMs alone the decode takes 57 us at 4096 x
    // 4096 x 4096 against 35 for a bf16 X, and the backward 126 instead of 111)
    if (e == cudaSuccess) e = run_db();
    SkinnyArgs sa{};
    sa.Mp = static_cast<int>(K);
    sa.ncols = sa.nout = sa.ld = r;
    sa.scale = 1.0f;
    sa.mode = modeA;
    sa.out = dA;
    sa.d_status = d_status;
    if (e == cudaSuccess)
      e = launch_skinny<true, true, false, true>(SkinnyMaps<false, true>{tdZ}, sa, static_cast<int>(M), Sa,
                                                 SkinnySecond{},
                                                 SkinnyA8{X8, X8_scales, static_cast<int>(M), static_cast<int>(K)}, s2);
  } else {
    if (e == cudaSuccess)
      e = dadb_ctas > 0
              ? run_rank_rows<true, true>(tXmn, tdZ, static_cast<int>(K), static_cast<int>(M), r, 1.0f, modeA,
                                          dA, r, dadb_ctas, d_status, s2)
              : run_skinny<true, true>(tXmn, tdZ, static_cast<int>(K), static_cast<int>(M), r, 1.0f, modeA, dA,
                                       r, Sa, d_status, s2);
    if (e == cudaSuccess) e = run_db();
  }
  const cudaError_t ej = fork.join();
  return e == cudaSuccess ? ej : e;
}

}  // namespace qnf4
