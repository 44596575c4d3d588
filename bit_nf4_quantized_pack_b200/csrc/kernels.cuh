// Launchers of the library's kernels and device helpers shared between
// translation units.  Internal to the library (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <utility>

#include "common.cuh"

namespace qnf4 {

// One-time set-up per device (kernel attributes, occupancy queries).
// cudaFuncSetAttribute acts on the current device only, so every device that
// runs a kernel gets its own run of `f(dev)`; a failed run is retried on the
// next call.  Safe when several host threads make their first calls at once.
constexpr int kMaxDevices = 64;
class DeviceOnce {
 public:
  template <typename F>
  cudaError_t run(F&& f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = f(dev);
    if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  std::mutex mu_;
  std::atomic<bool> done_[kMaxDevices] = {};
};

// The scale codebook T8 (see make_t8_table in common.cuh), one copy per
// translation unit in constant memory; build_t8 stages it in shared memory,
// where a warp's lookups of different codes do not serialize.
static __constant__ T8Table kT8Table = make_t8_table();

__device__ __forceinline__ void build_t8(float* t8 /*256*/) {
  for (int u = threadIdx.x; u < 256; u += blockDim.x) t8[u] = kT8Table.v[u];
}

// Launch with programmatic stream serialization (and, when cluster_y > 1, a
// thread-block cluster of 1 x cluster_y x 1).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t st, int cluster_y, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_y > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 1;
    attr[n].val.clusterDim.y = static_cast<unsigned>(cluster_y);
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same for a kernel whose CTA pairs share tensor-core products
// (cta_group::2): clusters of 2 x 1 x 1, the pair's CTAs adjacent in x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_pair(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// selftest.cu — a wait that nothing completes, bounded by limit_ns
cudaError_t launch_bounded_wait_selftest(int32_t* d_status, uint64_t limit_ns, cudaStream_t st);

// quantize.cu.  With double quantization the workspace holds, from its
// start: 256 exponent bins of the scales (2 KB), the counter of finished
// encoder CTAs, the call's token, the flag of its mean and the counter of
// claimed chunks, then (at kQuantizeWsHead) one fp32 scale per 64-block; CTA
// 0 of every call resets the head (any contents on entry).
constexpr size_t kQuantizeWsHead = 2304;
cudaError_t launch_quantize(const void* W, int dtype, int64_t numel, uint8_t* packed,
                            float* absmax_out, bool dq, uint8_t* code8, float* s2, float* offset,
                            void* ws, int32_t* d_status, cudaStream_t st, int num_sms,
                            int codebook = 0);
size_t quantize_workspace_bytes(int64_t numel, bool dq);
// Sharded quantization (blocks [b0, b1) of a tensor of numel_total elements;
// W_shard points at element b0 * 64).  begin: packed bytes and, without DQ,
// the scales go straight into the full-size state; with DQ the shard's
// scales and the exponent bins of their sums go to `ws` (same layout as the
// quantize workspace).  end: with the bins holding the sum over every shard,
// the offset and the scale codes and s2 of the shard's groups.
cudaError_t launch_quantize_shard_begin(const void* W_shard, int dtype, int64_t numel_total,
                                        int64_t b0, int64_t b1, uint8_t* packed, float* absmax_out,
                                        bool dq, void* ws, int32_t* d_status, cudaStream_t st,
                                        int num_sms, int codebook);
cudaError_t launch_quantize_shard_end(int64_t numel_total, int64_t b0, int64_t b1, const void* ws,
                                      uint8_t* code8, float* s2, float* offset, cudaStream_t st,
                                      int num_sms);

// dequantize.cu
cudaError_t launch_dequantize(const uint8_t* packed, int64_t numel, const float* absmax,
                              const uint8_t* code8, const float* s2, const float* offset,
                              uint16_t* out, int32_t* d_status, cudaStream_t st, int num_sms,
                              int codebook = 0);

// Decode-scale view of a quantized weight, shared by the GEMM and GEMV paths.
struct ScaleView {
  int codebook;          // 0: NF4, 1: uniform INT4 (its stored scale is amax / 7)
  const float* absmax;   // non-null when not double-quantized
  const uint8_t* code8;  // non-null when double-quantized
  const float* s2;
  const float* offset;
};

// merge.cu — the merged dense weight RN_bf16(ŵ + c·A·B)
cudaError_t launch_merge(int64_t K, int64_t N, int r, float c, ScaleView sv, const uint8_t* packed,
                         const uint16_t* A, const uint16_t* B, uint16_t* out, int32_t* d_status,
                         cudaStream_t st);

// gemv.cu — the M <= 16 forward (and, with zc_only, the recompute of its Zc):
// A_pad is A with its rows padded to rp (a multiple of 8) columns; Zc is
// written with row pitch ldz (columns r .. ldz-1 as 0) by one CTA.
struct GemvPlan {
  int G;     // 256-column groups
  int S;     // K splits = cluster size
  int per;   // 128-row stages per split
};
GemvPlan gemv_plan(int64_t K, int64_t N, int num_sms);
cudaError_t launch_gemv(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                        const uint8_t* packed, ScaleView sv, const uint16_t* A_pad, int rp,
                        const uint16_t* B, float c, uint16_t* Y, uint16_t* Zc, int ldz,
                        bool zc_only, int32_t* d_status, cudaStream_t st, int num_sms);

// linear.cu — work beside the caller's stream `st`, on a library-owned stream per
// device: fork, queue on `st` what goes first, enter, queue the work beside it on
// the stream that enter() gives, join.  That is `st` itself, so that the work runs
// in order behind the rest, where no fork is wanted or none can be had: no stream
// could be created, or it is part of a capture that `st` is not part of (a
// backward captured by another thread takes it in until that capture ends, and a
// wait across the border would fail and end the capture too).
struct SideStream;
class SideFork {
 public:
  SideFork(cudaStream_t st, bool wanted);
  cudaStream_t enter();
  // `st` waits for the work beside it.  Always called after enter(), so that nothing
  // on `st` can run ahead of work already queued.
  cudaError_t join();

 private:
  std::unique_lock<std::mutex> lock_;   // from the fork to the join: the stream and its events are shared
  cudaStream_t st_, side_;
  SideStream* ss_ = nullptr;            // null: in order
};
// Whether a backward's dX (M x K over N) is long enough to run its adapter
// gradients beside it on that stream.
inline bool worth_forking(int64_t M, int64_t K, int64_t N) {
  return static_cast<double>(M) * K * N >= 1e10;
}

// linear.cu — forward and backward of the layer
size_t linear_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r);
size_t linear_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r);
cudaError_t launch_linear_fwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                              const uint8_t* packed, ScaleView sv, const uint16_t* A,
                              const uint16_t* B, float c, uint16_t* Y, uint16_t* Zc, void* ws,
                              size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms);
cudaError_t launch_linear_bwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* dY,
                              const uint16_t* X, const uint16_t* Zc, const uint8_t* packed,
                              ScaleView sv, const uint16_t* A, const uint16_t* B, float c,
                              uint16_t* dX, void* dA, void* dB, void* ws, size_t ws_bytes,
                              int32_t* d_status, cudaStream_t st, int num_sms, bool grad_bf16 = false,
                              const int8_t* X8 = nullptr, const float* X8_scales = nullptr);
// (dA, dB are fp32, or bf16 with grad_bf16; with X8 the layer's input is an
// 8-bit checkpoint, X is null and Zc is not)

// act8.cu — 8-bit activation checkpoints
cudaError_t launch_act8_quantize(const uint16_t* X, int64_t numel, int8_t* codes, float* scales,
                                 int32_t* d_status, cudaStream_t st, int num_sms);
cudaError_t launch_act8_dequantize(const int8_t* codes, const float* scales, int64_t numel, uint16_t* X,
                                   cudaStream_t st, int num_sms);

// gated.cu — the gated block over two weights
struct GatedWeights {
  const uint8_t *packed_g, *packed_u;
  ScaleView sv_g, sv_u;
  const uint16_t *Ag, *Bg, *Au, *Bu;
  float c;
  int act;
};
// What the forward keeps for the backward: g and u in bf16 (G, U) or in 8 bits
// (G8, Gs, U8, Us), and the rank-r products; all null when nothing is kept.
struct GatedKept {
  uint16_t *G, *U;
  int8_t *G8, *U8;
  float *Gs, *Us;
  uint16_t *Zg, *Zu;
};
size_t gated_fwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r);
size_t gated_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N, int r);
cudaError_t launch_gated_fwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                             const GatedWeights& w, uint16_t* H, const GatedKept& kept, void* ws,
                             size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms);
cudaError_t launch_gated_bwd(int64_t M, int64_t K, int64_t N, int r, const uint16_t* dH,
                             const uint16_t* X, const int8_t* X8, const float* X8_scales,
                             const GatedWeights& w, const GatedKept& kept, uint16_t* dX, void* dAg,
                             void* dBg, void* dAu, void* dBu, bool grad_bf16, void* ws,
                             size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms);

// gated_rows.cu — the gated forward for few rows (see there)
bool gated_rows_fit(int64_t M, int64_t K, int64_t N);
size_t gated_rows_workspace_bytes(int64_t M, int64_t K, int64_t N, int r);
cudaError_t launch_gated_rows(int64_t M, int64_t K, int64_t N, int r, const uint16_t* X,
                              const GatedWeights& w, uint16_t* H, const GatedKept& kept, void* ws,
                              size_t ws_bytes, int32_t* d_status, cudaStream_t st);

// loss.cu — softmax cross entropy behind an NF4 head
size_t loss_fwd_workspace_bytes(int64_t M, int64_t N);
size_t loss_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N);
cudaError_t launch_loss_fwd(int64_t M, int64_t K, int64_t N, int64_t vocab, const uint16_t* X,
                            const uint8_t* packed, ScaleView sv, const int64_t* labels,
                            int64_t ignore_index, float* loss, float* lse, void* ws, size_t ws_bytes,
                            int32_t* d_status, cudaStream_t st, int num_sms);
cudaError_t launch_loss_bwd(int64_t M, int64_t K, int64_t N, int64_t vocab, const float* dloss,
                            const uint16_t* X, const float* lse, const uint8_t* packed, ScaleView sv,
                            const int64_t* labels, int64_t ignore_index, uint16_t* dX, void* ws,
                            size_t ws_bytes, int32_t* d_status, cudaStream_t st, int num_sms);

}  // namespace qnf4
