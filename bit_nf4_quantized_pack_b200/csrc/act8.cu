// 8-bit activation checkpoints: the codec (see act.cuh for its arithmetic).
//
// Both directions stream: 2 B + 1 B and a 64th of 4 B per element, so HBM
// bounds them (4096 x 11008, 138 MB, three matrices and three outputs in turn: quantize
// 24.1 us, 5.7 TB/s, and 20.7 where the outputs' memory is the same each time and stays in
// L2; dequantize 25.3 us, 5.5 TB/s).
// Quantize: four lanes share a block of 64, each with sixteen
// elements (two 16-byte loads, one 16-byte store), so that a block's scale is
// formed four times and its largest magnitude crosses lanes in two shuffles of
// packed 16-bit maxima (bf16 magnitudes order as integers, NaN and infinity
// above all finite values).
#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "profile.cuh"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kQUnroll = 2;
constexpr int kQPerSm = 4;   // blocks that an SM holds at 59 registers a thread (8: 4 % slower)

// `pieces` of sixteen elements, a multiple of 4
__global__ void __launch_bounds__(kThreads)
    act8_quantize_kernel(const uint4* __restrict__ X, int64_t pieces, uint4* __restrict__ codes,
                         float* __restrict__ scales, int32_t* d_status) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  bool bad = false;
  // a block's four lanes enter together; the warp leaves the loop together once
  // its first lane is past the end
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i0 - lane < pieces;
       i0 += stride * kQUnroll) {
    uint4 x[kQUnroll][2];
#pragma unroll
    for (int u = 0; u < kQUnroll; ++u) {
      const int64_t i = i0 + u * stride;
#pragma unroll
      for (int h = 0; h < 2; ++h) x[u][h] = i < pieces ? __ldcs(X + 2 * i + h) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kQUnroll; ++u) {
      const int64_t i = i0 + u * stride;
      const uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t top = max(m & 0xFFFFu, m >> 16);
      bad |= top >= 0x7F80u;
      const float s = act8_scale(__uint_as_float(top << 16));
      const float inv = act8_inverse(s);
      const uint4 o = act8_codes16(w, s, inv);
      if (i < pieces) {
        codes[i] = o;
        if ((lane & 3) == 0) scales[i >> 2] = s;
      }
    }
  }
  if (bad) raise_status(d_status, QLORA_ERR_NONFINITE);
}

__global__ void __launch_bounds__(kThreads)
    act8_dequantize_kernel(const uint2* __restrict__ codes, const float* __restrict__ scales,
                           int64_t pieces, uint4* __restrict__ X) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i0 < pieces;
       i0 += stride * kUnroll) {
    uint2 q[kUnroll];
    float s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * stride;
      q[u] = i < pieces ? __ldcs(codes + i) : make_uint2(0, 0);
      s[u] = i < pieces ? __ldg(scales + (i >> 3)) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * stride;
      float v[4], w[4];
      act8_values4(q[u].x, s[u], v);
      act8_values4(q[u].y, s[u], w);
      const uint32_t o[4] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(w[0], w[1]),
                             pack_bf16x2(w[2], w[3])};
      if (i < pieces) X[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

unsigned grid_for(int64_t pieces, int unroll, int num_sms, int per_sm) {
  const int64_t want = (pieces + kThreads * unroll - 1) / (kThreads * unroll);
  const int64_t most = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<unsigned>(want < most ? want : most);
}

}  // namespace

cudaError_t launch_act8_quantize(const uint16_t* X, int64_t numel, int8_t* codes, float* scales,
                                 int32_t* d_status, cudaStream_t st, int num_sms) {
  const int64_t pieces = numel / 16;
  cudaError_t e;
  {
    ProfScope prof(kProfAct8, st);
    e = launch_pdl(act8_quantize_kernel, dim3(grid_for(pieces, kQUnroll, num_sms, kQPerSm)), dim3(kThreads), 0, st, 1,
                   reinterpret_cast<const uint4*>(X), pieces, reinterpret_cast<uint4*>(codes), scales,
                   d_status);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_act8_dequantize(const int8_t* codes, const float* scales, int64_t numel, uint16_t* X,
                                   cudaStream_t st, int num_sms) {
  const int64_t pieces = numel / 8;
  cudaError_t e;
  {
    ProfScope prof(kProfAct8, st);
    e = launch_pdl(act8_dequantize_kernel, dim3(grid_for(pieces, kUnroll, num_sms, 8)), dim3(kThreads), 0, st, 1,
                   reinterpret_cast<const uint2*>(codes), scales, pieces, reinterpret_cast<uint4*>(X));
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qnf4
