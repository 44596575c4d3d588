// Softmax cross entropy behind an NF4 frozen head (K x N, the vocabulary its
// first `vocab` columns), in pieces of the vocabulary, without the logits ever
// reaching memory:
//
//   l = X·Ŵ,  lse_i = log Σ_v exp(l_iv),  loss_i = lse_i - l_i[y_i]
//   dX_i = dloss_i (Σ_v softmax(l_i)_v Ŵ_v - Ŵ_{y_i})
//
// Forward: the fused GEMM's epilogue reduces each 128 columns of a row to
// their maximum and sum of exponentials (kModeLossStats); a second kernel joins
// those.  Backward: per piece of columns the logits are formed again and the
// epilogue writes P = bf16(exp(l - lse) - onehot) (kModeLossGrad); a fused GEMM
// adds dloss·(P·Ŵᵀ) to the fp32 sums of the pieces before (kModeLossDX).  A
// piece holds at most about 2^26 elements of P (128 MB): 4096 rows over 32001
// tokens took 5 % longer in pieces of half that (more partial waves of tiles) and
// 8 % less in one piece (which would keep what the logits take).
//
// Roundings: the logits are fp32 sums in the tensor cores, which cut each addition
// towards zero (loss and lse 5e-6 from 64 bits at K = 8192); maximum, sum of
// exponentials, softmax - onehot and the pieces' sums are fp32; P is bf16 because it is
// an operand of the product with Ŵᵀ (dX 1.7e-3 to 1.9e-3 of its norm from 64 bits,
// its own rounding 1.7e-3).
//
// Bound: the tensor pipe and the power cap.  4096 x 4096 x 32001, forward and backward:
// 2607 us (1.23 PFLOP/s over the three products that run), of which statistics 570
// and per piece of 16128 columns the logits again about 390 and dX 375; forward
// alone, 512 x 8192 x 65536, 456 us (1.21).
// dX splits its contraction where it has few tiles and the vocabulary is one piece.
// With several pieces it does not: 2048 x 512 over 65536 tokens (two pieces, 8 tiles
// for 74 pairs) takes 883 us backward beside 205 forward, where 4096 x 4096 over
// 32001 (128 tiles) takes 1570 beside 723.
#include "common.cuh"
#include "fused.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "rank.cuh"
#include "tmap.cuh"

namespace qnf4 {
namespace {

constexpr int64_t kPieceElems = 1ll << 26;

// Columns of a piece: pieces of equal width, a multiple of 256.
int64_t piece_cols(int64_t M, int64_t N) {
  const int64_t most = kPieceElems / M > 256 ? kPieceElems / M : 256;
  const int64_t n = (N + most - 1) / most;
  const int64_t per = (N + n - 1) / n;
  return (per + 255) / 256 * 256;
}

// Joins the (maximum, sum) pairs of a row: 32 rows x 8 slices of the pairs per
// block.
constexpr int kJoinRows = 32, kJoinSlices = 8;
__global__ void __launch_bounds__(kJoinRows * kJoinSlices)
    loss_join_kernel(const float2* __restrict__ stats, const float* __restrict__ label_logit, int M,
                     int nstats, int64_t vocab, const int64_t* __restrict__ labels, int64_t ignore_index,
                     float* __restrict__ loss, float* __restrict__ lse, int32_t* d_status) {
  __shared__ float sm[kJoinSlices][kJoinRows], ss[kJoinSlices][kJoinRows];
  pdl_launch_dependents();
  pdl_wait();
  const int rl = threadIdx.x % kJoinRows, sl = threadIdx.x / kJoinRows;
  const int row = blockIdx.x * kJoinRows + rl;
  float m = -CUDART_INF_F, s = 0.0f;
  auto add = [&](float m2, float s2) {
    if (m2 == -CUDART_INF_F && s2 == 0.0f) return;   // no column
    const float nm = fmaxf(m, m2);
    s = (m == nm ? s : s * ex2((m - nm) * kLog2E)) + (m2 == nm ? s2 : s2 * ex2((m2 - nm) * kLog2E));
    m = nm;
  };
  if (row < M)
    for (int t = sl; t < nstats; t += kJoinSlices) {
      const float2 p = stats[static_cast<int64_t>(t) * M + row];
      add(p.x, p.y);
    }
  sm[sl][rl] = m;
  ss[sl][rl] = s;
  __syncthreads();
  if (sl != 0 || row >= M) return;
  m = -CUDART_INF_F;
  s = 0.0f;
  for (int k = 0; k < kJoinSlices; ++k) add(sm[k][rl], ss[k][rl]);
  const float v = m + logf(s);
  lse[row] = v;
  const int64_t y = labels[row];
  float out = 0.0f;
  if (y != ignore_index) {
    if (y < 0 || y >= vocab)
      raise_status(d_status, QLORA_ERR_INVALID_ARG);
    else
      out = v - label_logit[row];
  }
  loss[row] = out;
}

LossArgs loss_args(int64_t M, int64_t N, int64_t vocab, const uint8_t* packed, ScaleView sv,
                   const int64_t* labels, int64_t ignore_index, int32_t* d_status) {
  LossArgs a{};
  a.M = static_cast<int>(M);
  a.Nw = static_cast<int>(N);
  a.m_tiles = static_cast<int>((M + kFPairRows - 1) / kFPairRows);
  a.sv = sv;
  a.packed = packed;
  a.vocab = static_cast<int>(vocab);
  a.labels = labels;
  a.ignore_index = ignore_index;
  a.d_status = d_status;
  return a;
}

template <int kMode>
cudaError_t run_loss(const CUtensorMap& act, const CUtensorMap& out, LossArgs a, int nk, int64_t cols, cudaStream_t st,
                     int num_sms, uint16_t* dX = nullptr) {
  cudaError_t e = set_fused_attr<kMode>();
  if (e != cudaSuccess) return e;
  a.nk = nk;
  a.Nout = static_cast<int>(cols);
  a.n_tiles = static_cast<int>((cols + kFPairCols - 1) / kFPairCols);
  if constexpr (kMode == kModeLossDX)
    set_split(a, a.part);
  else
    set_rows(a);
  const int items = a.m_tiles * a.n_tiles * (kMode == kModeLossDX ? a.splits : 1);
  {
    ProfScope prof(kProfLoss, st);
    e = launch_pdl_pair(fused_nf4_gemm_kernel<kMode>, dim3(2 * fused_pairs(items, num_sms)), dim3(kFThreads), kFSmem,
                        st, typename ModeTypes<kMode>::Maps{act, out}, a);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (kMode == kModeLossDX && e == cudaSuccess && a.splits > 1) e = launch_split_join(a, dX, kProfLoss, st);
  return e;
}

}  // namespace

size_t loss_fwd_workspace_bytes(int64_t M, int64_t N) {
  return align256(static_cast<size_t>((N + kFPairCols - 1) / kFPairCols * 2) * M * sizeof(float2)) +
         align256(static_cast<size_t>(M) * 4);
}

size_t loss_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  const int64_t per = piece_cols(M, N);
  // P; the pieces' sums, or with one piece a split dX's
  return align256(static_cast<size_t>(M) * per * 2) +
         (per < N ? align256(static_cast<size_t>(M) * K * 4) : split_bytes(M, K, N / 64));
}

cudaError_t launch_loss_fwd(int64_t M, int64_t K, int64_t N, int64_t vocab, const uint16_t* X,
                            const uint8_t* packed, ScaleView sv, const int64_t* labels,
                            int64_t ignore_index, float* loss, float* lse, void* ws, size_t ws_bytes,
                            int32_t* d_status, cudaStream_t st, int num_sms) {
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  // only the tiles that hold columns of the vocabulary
  const int n_tiles = static_cast<int>((vocab + kFPairCols - 1) / kFPairCols);
  float2* stats = static_cast<float2*>(cur.take(static_cast<size_t>(2 * n_tiles) * M * sizeof(float2)));
  float* lab = static_cast<float*>(cur.take(static_cast<size_t>(M) * 4));
  if (!cur.ok) return cudaErrorInvalidValue;
  CUtensorMap tX;
  if (!make_tmap_2d(&tX, X, kBF16, 2, M, K, K, 64, 128, kSW128)) return cudaErrorInvalidValue;
  LossArgs a = loss_args(M, N, vocab, packed, sv, labels, ignore_index, d_status);
  a.stats = stats;
  a.label_logit = lab;
  const int64_t cols = static_cast<int64_t>(n_tiles) * kFPairCols < N ? static_cast<int64_t>(n_tiles) * kFPairCols : N;
  cudaError_t e = run_loss<kModeLossStats>(tX, tX, a, static_cast<int>(K / 64), cols, st, num_sms);
  if (e != cudaSuccess) return e;
  {
    ProfScope prof(kProfLoss, st);
    e = launch_pdl(loss_join_kernel, dim3(static_cast<unsigned>((M + kJoinRows - 1) / kJoinRows)),
                   dim3(kJoinRows * kJoinSlices), 0, st, 1, static_cast<const float2*>(stats),
                   static_cast<const float*>(lab), static_cast<int>(M), 2 * n_tiles, vocab, labels,
                   ignore_index, loss, lse, d_status);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_loss_bwd(int64_t M, int64_t K, int64_t N, int64_t vocab, const float* dloss,
                            const uint16_t* X, const float* lse, const uint8_t* packed, ScaleView sv,
                            const int64_t* labels, int64_t ignore_index, uint16_t* dX, void* ws,
                            size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms) {
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  const int64_t per = piece_cols(M, N);
  uint16_t* P = static_cast<uint16_t*>(cur.take(static_cast<size_t>(M) * per * 2));
  float* acc = per < N ? static_cast<float*>(cur.take(static_cast<size_t>(M) * K * 4)) : nullptr;
  // (split by the vocabulary's steps, which are no more than the head's)
  const size_t split = per < N ? 0 : split_bytes(M, K, (vocab + 63) / 64);
  float* part = split > 0 ? static_cast<float*>(cur.take(split)) : nullptr;
  if (!cur.ok) return cudaErrorInvalidValue;
  CUtensorMap tX;
  if (!make_tmap_2d(&tX, X, kBF16, 2, M, K, K, 64, 128, kSW128)) return cudaErrorInvalidValue;
  CUtensorMap tdX;
  if (!make_tmap_2d(&tdX, dX, kBF16, 2, M, K, K, 32, 32, kSW64)) return cudaErrorInvalidValue;
  // whole 64-blocks of the vocabulary; the head's columns behind them add nothing
  const int64_t end = (vocab + 63) / 64 * 64;
  for (int64_t c0 = 0; c0 < end; c0 += per) {
    const int64_t cols = end - c0 < per ? end - c0 : per;
    LossArgs a = loss_args(M, N, vocab, packed, sv, labels, ignore_index, d_status);
    a.col0 = static_cast<int>(c0);
    a.lse = lse;
    a.dloss = dloss;
    CUtensorMap tPout;
    if (!make_tmap_2d(&tPout, P, kBF16, 2, M, cols, cols, 32, 32, kSW64)) return cudaErrorInvalidValue;
    cudaError_t e = run_loss<kModeLossGrad>(tX, tPout, a, static_cast<int>(K / 64), cols, st, num_sms);
    if (e != cudaSuccess) return e;
    CUtensorMap tP;
    if (!make_tmap_2d(&tP, P, kBF16, 2, M, cols, cols, 64, 128, kSW128)) return cudaErrorInvalidValue;
    a.part = part;
    a.acc = acc;
    a.first = c0 == 0 ? 1 : 0;
    a.last = c0 + cols >= end ? 1 : 0;
    e = run_loss<kModeLossDX>(tP, tdX, a, static_cast<int>(cols / 64), K, st, num_sms, dX);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qnf4
