// The gated block over two NF4 frozen-base weights with LoRA adapters:
//
//   g = X·Ŵg + Zg·Bg,  u = X·Ŵu + Zu·Bu,  H = act(g) * u,   Z = bf16(c·X·A)
//   dG = dH * u * act'(g),  dU = dH * act(g),  dZ = bf16(c·d·Bᵀ),
//   dX = dG·Ŵgᵀ + dU·Ŵuᵀ + dZg·Agᵀ + dZu·Auᵀ,  dA = Xᵀ·dZ,  dB = Zᵀ·d
//
// Z and dZ are bf16 as in the layer: summed in fp32, they are operands of the products
// behind them.  Forward: the rank-r products of both adapters in one launch, before or beside one
// fused GEMM over both weights whose epilogue forms H (and keeps g and u, in bf16 or
// in 8 bits).  Backward: one pass over dH, g and u for dG and dU, both dZ in
// one launch, one fused GEMM over both weights for dX, and beside it both dA
// and both dB in a launch each.
//
// At 4096 x 4096 x 11008, rank 64, keeping g and u: forward 26 us of rank-r products
// and 552 of the fused GEMM, backward 83 for dG and dU and about 520 for dX with
// dZ, dA and dB beside it: 1.44 PFLOP/s in dX, 1.34 in the forward, whose ten waves
// of tiles hold 9.3.
#include "act.cuh"
#include "common.cuh"
#include "fused.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "rank.cuh"
#include "tmap.cuh"

namespace qnf4 {
namespace {

// dG and dU of eight elements a thread, in fp32 up to one rounding to bf16: they are
// operands of three tensor-core products each (dX, dZ, dB), which take 16 bits, and a
// pair of bf16 operands for the two halves of an fp32 value would double those
// products.  With it the gradients are 3.5e-3 of their norm from 64 bits where the
// result's own rounding is 1.7e-3.  kG8: g and u come as 8-bit
// checkpoints.  Streams 10 (8-bit: 8.1) bytes an element: HBM-bound, 83 us at 4096 x
// 11008 (451 MB, 5.4 TB/s).
template <bool kG8>
__global__ void __launch_bounds__(256)
    gated_grad_kernel(const uint4* __restrict__ dH, const void* __restrict__ G, const void* __restrict__ U,
                      const float* __restrict__ Gs, const float* __restrict__ Us, int64_t pieces, int act,
                      uint4* __restrict__ dG, uint4* __restrict__ dU) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += stride) {
    const uint4 h4 = __ldcs(dH + i);
    float g[8], u[8];
    if constexpr (kG8) {
      const uint2 g2 = __ldcs(static_cast<const uint2*>(G) + i), u2 = __ldcs(static_cast<const uint2*>(U) + i);
      const float sg = __ldg(Gs + (i >> 3)), su = __ldg(Us + (i >> 3));
      const uint32_t gw[2] = {g2.x, g2.y}, uw[2] = {u2.x, u2.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float vg[4], vu[4];
        act8_values4(gw[k], sg, vg);
        act8_values4(uw[k], su, vu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[4 * k + j] = round_bf16(vg[j]);
          u[4 * k + j] = round_bf16(vu[j]);
        }
      }
    } else {
      const uint4 g4 = __ldcs(static_cast<const uint4*>(G) + i), u4 = __ldcs(static_cast<const uint4*>(U) + i);
      const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        g[2 * k] = __uint_as_float(gw[k] << 16);
        g[2 * k + 1] = __uint_as_float(gw[k] & 0xFFFF0000u);
        u[2 * k] = __uint_as_float(uw[k] << 16);
        u[2 * k + 1] = __uint_as_float(uw[k] & 0xFFFF0000u);
      }
    }
    const uint32_t hw[4] = {h4.x, h4.y, h4.z, h4.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float d0, d1;
      const float h0 = __uint_as_float(hw[k] << 16), h1 = __uint_as_float(hw[k] & 0xFFFF0000u);
      const float a0 = act_value_grad(act, g[2 * k], d0), a1 = act_value_grad(act, g[2 * k + 1], d1);
      og[k] = pack_bf16x2(h0 * u[2 * k] * d0, h1 * u[2 * k + 1] * d1);
      ou[k] = pack_bf16x2(h0 * a0, h1 * a1);
    }
    dG[i] = make_uint4(og[0], og[1], og[2], og[3]);
    dU[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// Two rank-r contractions in one launch (see run_skinny for the modes).
template <bool kAmn, bool kBmn>
cudaError_t run_skinny_two(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ta2,
                           const CUtensorMap& tb2, int Mp, int Kp, int ncols, float scale, int mode,
                           void* out, void* out_second, int ld, int32_t* d_status, cudaStream_t st,
                           int nout, uint16_t* pad = nullptr, uint16_t* pad_second = nullptr, int ld2 = 0) {
  SkinnyArgs a{};
  a.Mp = Mp;
  a.ncols = ncols;
  a.nout = nout;
  a.scale = scale;
  a.mode = mode;
  a.out = out;
  a.ld = ld;
  a.out2 = pad;
  a.ld2 = ld2;
  a.d_status = d_status;
  // half of the sizing SM count for each of the two
  const int splits = skinny_splits(Mp, (Kp + 63) / 64, g_ws_sms / 2);
  return launch_skinny<kAmn, kBmn, true, false>(SkinnyMaps<true, false>{ta, tb, ta2, tb2}, a, Kp, splits,
                                                SkinnySecond{out_second, pad_second}, SkinnyA8{}, st);
}

// Two rank-r products X·A or G·Bᵀ on the SMs that the fused GEMM leaves free.
template <bool kAmn, bool kBmn>
cudaError_t run_rank_rows_two(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ta2,
                              const CUtensorMap& tb2, int Mp, int Kp, int ncols, float scale, void* out,
                              void* out_second, int ld, int ctas, int32_t* d_status, cudaStream_t st, int nout,
                              uint16_t* pad = nullptr, uint16_t* pad_second = nullptr, int ld2 = 0) {
  SkinnyArgs a{};
  a.Mp = Mp;
  a.ncols = ncols;
  a.nout = nout;
  a.scale = scale;
  a.out = out;
  a.ld = ld;
  a.out2 = pad;
  a.ld2 = ld2;
  a.d_status = d_status;
  return launch_rank_rows<kAmn, kBmn, true>(SkinnyMaps<true, false>{ta, tb, ta2, tb2}, a, Kp, ctas,
                                            SkinnySecond{out_second, pad_second}, st);
}

int tiles_of(int64_t n, int per) { return static_cast<int>((n + per - 1) / per); }

// SMs that the fused GEMM of `tiles` tiles of `nk` K-steps leaves free, or 0 where
// two rank-r products over M rows of `cols` columns would not be done there about
// when its first tile comes to the LoRA steps: a CTA streams about 58 KB a us and
// loses two at a tile's start and end, a K-step takes 0.55 to 0.75 us.  Against both
// products split over all SMs before it, the forward back to back (alone between
// other work 1000 x 4096 x 11008 takes 166 us): 45.2 and 48.4 us at 333 x 4096 x
// 4096, 54.5 and 58.7 at 700 x 4096 x 4096, 143 and 149 at 1000 x 4096 x 11008, 199 and
// 205 at 1500 x 4096 x 11008; beyond the limit 97.4 and 95.2 at 2048 x 2048 x 5632.
int free_sms_for_two(int64_t M, int64_t cols, int tiles, int nk) {
  const int sms = rank_rows_ctas(0.0, tiles, 1.0);
  if (sms == 0) return 0;
  const int rounds = tiles_of(2 * tiles_of(M, 128), sms);
  return rounds * (256.0 * cols + 0.1e6) <= 0.037e6 * nk ? sms : 0;
}

}  // namespace

size_t gated_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r) {
  if (gated_rows_fit(M, K, N)) return gated_rows_workspace_bytes(M, K, N, r);
  const int rp = padded_rank(r);
  // Zg and Zu (a copy padded to rp columns where the caller keeps them with r),
  // and both A padded to rp columns when r is not a multiple of 8
  return 2 * align256(static_cast<size_t>(M) * rp * 2) +
         (rp != r ? 2 * align256(static_cast<size_t>(K) * rp * 2) : 0);
}

size_t gated_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r) {
  const int rp = padded_rank(r);
  // dG, dU; dZg, dZu; a split dX's sums; when r is not a multiple of 8 padded
  // copies of Zg, Zu, Ag, Au
  return split_bytes(M, K, 2 * (N / 64)) + 2 * align256(static_cast<size_t>(M) * N * 2) + 2 * align256(static_cast<size_t>(M) * rp * 2) +
         (rp != r ? 2 * align256(static_cast<size_t>(M) * rp * 2) + 2 * align256(static_cast<size_t>(K) * rp * 2)
                  : 0);
}

cudaError_t launch_gated_fwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                             const GatedWeights& w, uint16_t* H, const GatedKept& kept, void* ws,
                             size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms) {
  // up to 128 rows: 73 us there against 79 for 129 here at 4096 x 11008 (and 35
  // against 79 for one row)
  if (gated_rows_fit(M, K, N)) return launch_gated_rows(M, K, N, r, X, w, H, kept, ws, ws_bytes, d_status, st);
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  const int rp = padded_rank(r);
  const bool pad = rp != r;
  const int iM = static_cast<int>(M), iK = static_cast<int>(K);
  uint16_t* Zwg = static_cast<uint16_t*>(cur.take(static_cast<size_t>(M) * rp * 2));
  uint16_t* Zwu = static_cast<uint16_t*>(cur.take(static_cast<size_t>(M) * rp * 2));
  uint16_t* Apg = pad ? static_cast<uint16_t*>(cur.take(static_cast<size_t>(K) * rp * 2)) : nullptr;
  uint16_t* Apu = pad ? static_cast<uint16_t*>(cur.take(static_cast<size_t>(K) * rp * 2)) : nullptr;
  if (!cur.ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  const uint16_t *Ag = w.Ag, *Au = w.Au;
  if (pad) {
    e = launch_pad_sets(PadSet{{w.Ag, w.Au}, {Apg, Apu}, {K, K}}, 2, r, rp, st);
    if (e != cudaSuccess) return e;
    Ag = Apg;
    Au = Apu;
  }
  // Z: into the kept buffers (M x r) when there are, with a copy of row pitch
  // rp for the fused kernel's TMA where r is not a multiple of 8
  const bool keep = kept.Zg != nullptr;
  uint16_t *Zg = keep ? kept.Zg : Zwg, *Zu = keep ? kept.Zu : Zwu;
  const bool copy = keep && pad;
  CUtensorMap tX, tAg, tAu;
  if (!make_tmap_2d(&tX, X, kBF16, 2, M, K, K, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tAg, Ag, kBF16, 2, K, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tAu, Au, kBF16, 2, K, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  e = set_fused_attr<kModeGatedFwd>();
  if (e != cudaSuccess) return e;
  ModeTypes<kModeGatedFwd>::Maps maps;
  maps.act = tX;
  maps.act2 = tX;
  if (!make_tmap_2d(&maps.la, copy ? Zwg : Zg, kBF16, 2, M, rp, rp, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.la2, copy ? Zwu : Zu, kBF16, 2, M, rp, rp, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.lb, w.Bg, kBF16, 2, r, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.lb2, w.Bu, kBF16, 2, r, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.out, H, kBF16, 2, M, N, N, 32, 32, kSW64)) return cudaErrorInvalidValue;
  maps.g = maps.u = maps.out;
  if (kept.G != nullptr) {
    if (!make_tmap_2d(&maps.g, kept.G, kBF16, 2, M, N, N, 32, 32, kSW64)) return cudaErrorInvalidValue;
    if (!make_tmap_2d(&maps.u, kept.U, kBF16, 2, M, N, N, 32, 32, kSW64)) return cudaErrorInvalidValue;
  } else if (kept.G8 != nullptr) {
    if (!make_tmap_2d(&maps.g, kept.G8, kU8, 1, M, N, N, 64, 32, kSW64)) return cudaErrorInvalidValue;
    if (!make_tmap_2d(&maps.u, kept.U8, kU8, 1, M, N, N, 64, 32, kSW64)) return cudaErrorInvalidValue;
  }
  GatedArgs ga{};
  ga.M = iM;
  ga.Nout = static_cast<int>(N);
  ga.Nw = static_cast<int>(N);
  ga.nk = static_cast<int>(K / 64);
  ga.rsteps = rsteps_of(r);
  ga.n_tiles = tiles_of(N, mode_tile_cols(kModeGatedFwd));
  set_rows(ga);
  ga.sv = w.sv_g;
  ga.packed = w.packed_g;
  ga.sv2 = w.sv_u;
  ga.packed2 = w.packed_u;
  ga.act = w.act;
  ga.keep = kept.G != nullptr ? 1 : (kept.G8 != nullptr ? 2 : 0);
  ga.Gs = kept.Gs;
  ga.Us = kept.Us;
  ga.d_status = d_status;
  // Z beside the fused GEMM where it leaves SMs free for long enough, else split
  // over all SMs before it
  const int free_sms = free_sms_for_two(M, K, ga.m_tiles * ga.n_tiles, ga.nk);
  const int zld = keep ? r : rp;
  uint16_t *pad_g = copy ? Zwg : nullptr, *pad_u = copy ? Zwu : nullptr;
  if (free_sms > 0)
    e = run_rank_rows_two<false, true>(tX, tAg, tX, tAu, iM, iK, rp, w.c, Zg, Zu, zld, free_sms, d_status, st, zld,
                                       pad_g, pad_u, rp);
  else
    e = run_skinny_two<false, true>(tX, tAg, tX, tAu, iM, iK, rp, w.c, 0, Zg, Zu, zld, d_status, st, zld, pad_g,
                                    pad_u, rp);
  if (e != cudaSuccess) return e;
  const int grid = fused_pairs(ga.m_tiles * ga.n_tiles, num_sms);
  {
    ProfScope prof(kProfGated, st);
    e = launch_pdl_pair(fused_nf4_gemm_kernel<kModeGatedFwd>, dim3(2 * grid), dim3(kFThreads),
                        kFSmem, st, maps, ga);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_gated_bwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* dH,
                             const uint16_t* X, const int8_t* X8, const float* X8_scales,
                             const GatedWeights& w, const GatedKept& kept, uint16_t* dX, void* dAg,
                             void* dBg, void* dAu, void* dBu, bool grad_bf16, void* ws,
                             size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms) {
  WsCursor cur{static_cast<char*>(ws), ws_bytes};
  const int rp = padded_rank(r);
  const bool pad = rp != r;
  const int iM = static_cast<int>(M), iK = static_cast<int>(K), iN = static_cast<int>(N);
  auto bf16_rows = [&](int64_t rows, int64_t cols) {
    return static_cast<uint16_t*>(cur.take(static_cast<size_t>(rows) * cols * 2));
  };
  uint16_t *dG = bf16_rows(M, N), *dU = bf16_rows(M, N);
  uint16_t *dZg = bf16_rows(M, rp), *dZu = bf16_rows(M, rp);
  uint16_t *Zpg = nullptr, *Zpu = nullptr, *Apg = nullptr, *Apu = nullptr;
  if (pad) {
    Zpg = bf16_rows(M, rp);
    Zpu = bf16_rows(M, rp);
    Apg = bf16_rows(K, rp);
    Apu = bf16_rows(K, rp);
  }
  const size_t split = split_bytes(M, K, 2 * (N / 64));
  float* part = split > 0 ? static_cast<float*>(cur.take(split)) : nullptr;
  if (!cur.ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  const uint16_t *Ag = w.Ag, *Au = w.Au, *Zg = kept.Zg, *Zu = kept.Zu;
  if (pad) {
    e = launch_pad_sets(PadSet{{w.Ag, w.Au, kept.Zg, kept.Zu}, {Apg, Apu, Zpg, Zpu}, {K, K, M, M}}, 4, r, rp, st);
    if (e != cudaSuccess) return e;
    Ag = Apg;
    Au = Apu;
    Zg = Zpg;
    Zu = Zpu;
  }
  // dG, dU
  {
    const int64_t pieces = M * N / 8;
    const int64_t want = (pieces + 255) / 256, most = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    ProfScope prof(kProfGated, st);
    const bool g8 = kept.G8 != nullptr;
    e = launch_pdl(g8 ? gated_grad_kernel<true> : gated_grad_kernel<false>, grid, dim3(256), 0, st, 1,
                   reinterpret_cast<const uint4*>(dH),
                   g8 ? static_cast<const void*>(kept.G8) : static_cast<const void*>(kept.G),
                   g8 ? static_cast<const void*>(kept.U8) : static_cast<const void*>(kept.U),
                   static_cast<const float*>(kept.Gs), static_cast<const float*>(kept.Us), pieces, w.act,
                   reinterpret_cast<uint4*>(dG), reinterpret_cast<uint4*>(dU));
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // dX over both weights, after dZ (see below)
  CUtensorMap tG, tU, tBg, tBu;
  if (!make_tmap_2d(&tG, dG, kBF16, 2, M, N, N, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tU, dU, kBF16, 2, M, N, N, 64, 128, kSW128)) return cudaErrorInvalidValue;
  e = set_fused_attr<kModeGatedBwd>();
  if (e != cudaSuccess) return e;
  ModeTypes<kModeGatedBwd>::Maps maps;
  maps.act = tG;
  maps.act2 = tU;
  if (!make_tmap_2d(&maps.la, dZg, kBF16, 2, M, rp, rp, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.la2, dZu, kBF16, 2, M, rp, rp, 64, 128, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.lb, Ag, kBF16, 2, K, rp, rp, 64, kFBN, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.lb2, Au, kBF16, 2, K, rp, rp, 64, kFBN, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&maps.out, dX, kBF16, 2, M, K, K, 32, 32, kSW64)) return cudaErrorInvalidValue;
  GatedArgs ga{};
  ga.M = iM;
  ga.Nout = iK;
  ga.Nw = iN;
  ga.nk = static_cast<int>(2 * (N / 64));
  ga.rsteps = rsteps_of(r);
  ga.m_tiles = tiles_of(M, kFPairRows);
  ga.n_tiles = tiles_of(K, mode_tile_cols(kModeGatedBwd));
  ga.sv = w.sv_g;
  ga.packed = w.packed_g;
  ga.sv2 = w.sv_u;
  ga.packed2 = w.packed_u;
  ga.d_status = d_status;
  set_split(ga, part);
  // dZ = bf16(c d Bᵀ), both (columns past r are zero: B's rows past r arrive as zero fill)
  if (!make_tmap_2d(&tBg, w.Bg, kBF16, 2, r, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tBu, w.Bu, kBF16, 2, r, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  // On the SMs that dX leaves free, beside it, or over all SMs before it; always so
  // where dX is split (its items come to the LoRA steps soon).  The backward so and
  // so: 260 and 269 us at 1500 x 4096 x 11008, 632 and 640 at 4096 x 4096 x 11008, 1004
  // and 1047 at 4096 x 5120 x 13824; split, 88 and 86 at 700 x 4096 x 4096.
  const int free_sms = ga.splits > 1 ? 0 : free_sms_for_two(M, N, ga.m_tiles * ga.n_tiles, ga.nk);
  if (free_sms > 0)
    e = run_rank_rows_two<false, false>(tG, tBg, tU, tBu, iM, iN, rp, w.c, dZg, dZu, rp, free_sms, d_status, st, rp);
  else
    e = run_skinny_two<false, false>(tG, tBg, tU, tBu, iM, iN, rp, w.c, 0, dZg, dZu, rp, d_status, st, rp);
  if (e != cudaSuccess) return e;
  const int grid = fused_pairs(ga.m_tiles * ga.n_tiles * ga.splits, num_sms);
  // operands of dA and dB, read transposed
  CUtensorMap tXmn, tdZg, tdZu, tGmn, tUmn, tZg, tZu;
  if (X8 == nullptr && !make_tmap_2d(&tXmn, X, kBF16, 2, M, K, K, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tdZg, dZg, kBF16, 2, M, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tdZu, dZu, kBF16, 2, M, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tGmn, dG, kBF16, 2, M, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tUmn, dU, kBF16, 2, M, N, N, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tZg, Zg, kBF16, 2, M, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;
  if (!make_tmap_2d(&tZu, Zu, kBF16, 2, M, rp, rp, 64, 64, kSW128)) return cudaErrorInvalidValue;

  // dX first, then dA and dB (which need only dZ, Z, X, dG and dU) on the
  // library's stream, so that they take the SMs dX leaves idle; the caller's
  // stream waits for them before the call returns.  Small steps run in order:
  // the fork and the join cost more than they hide (the whole step at 333 x 1088
  // x 2752 100 us forked, 89 in order; at 700 x 4096 x 4096 158 and 159; at 1500 x
  // 4096 x 11008 500 and 533).
  SideFork fork(st, !prof_timing(kProfSkinny) && worth_forking(M, K, N));
  {
    ProfScope prof(kProfGated, st);
    e = launch_pdl_pair(fused_nf4_gemm_kernel<kModeGatedBwd>, dim3(2 * grid), dim3(kFThreads), kFSmem, st,
                        maps, ga);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess && ga.splits > 1) e = launch_split_join(ga, dX, kProfGated, st);
  const cudaStream_t s2 = fork.enter();
  if (e == cudaSuccess && X8 != nullptr) {
    SkinnyArgs sa{};
    sa.Mp = iK;
    sa.ncols = sa.nout = sa.ld = r;
    sa.scale = 1.0f;
    sa.mode = grad_bf16 ? 0 : 1;
    sa.out = dAg;
    sa.d_status = d_status;
    e = launch_skinny<true, true, true, true>(SkinnyMaps<true, true>{tdZg, tdZu}, sa, iM,
                                              skinny_splits(iK, (iM + 63) / 64, g_ws_sms / 2),
                                              SkinnySecond{dAu, nullptr}, SkinnyA8{X8, X8_scales, iM, iK}, s2);
  } else if (e == cudaSuccess) {
    e = run_skinny_two<true, true>(tXmn, tdZg, tXmn, tdZu, iK, iM, r, 1.0f, grad_bf16 ? 0 : 1, dAg, dAu, r,
                                   d_status, s2, r);
  }
  if (e == cudaSuccess)
    e = run_skinny_two<true, true>(tGmn, tZg, tUmn, tZu, iN, iM, r, 1.0f, grad_bf16 ? 3 : 2, dBg, dBu, r,
                                   d_status, s2, r);
  const cudaError_t ej = fork.join();
  return e == cudaSuccess ? ej : e;
}

}  // namespace qnf4
