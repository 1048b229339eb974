// layers.h - interfaces between the ABI of dyra_layers.h (layers_api.cu) and
// its kernels.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "dyra_layers.h"
#include "internal.h"

namespace dyra {

// Every kernel of the layers is a programmatic dependent launch: its grid may be
// set up while the one before it in the stream still runs, whichever kernel that
// is, and waits for it (griddepcontrol.wait) before it reads or writes memory. The
// wait is for the whole grid before, which waited for its own predecessor, so the
// order of the stream holds. Calls that follow one another hide their launches
// behind each other in this way.
// One exception: the experts' down kernel (StreamCommon::late_b) reads the ids and
// weights and copies Wd before its wait. It may, because the gate-up kernel, always
// the one before it, lets it start only after its own wait is over: whatever wrote
// those is complete then. Most other kernels here let the next one start at once, so
// no other kernel may come between the two, and none may read before its wait
// behind a grid that does so.
template <class Kernel, class... Args>
inline int launch_dependent(Kernel kfn, dim3 grid, dim3 block, uint32_t smem, int cluster,
                            cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kfn, args...) == cudaSuccess ? 0 : -1;
}

// One matrix product with its epilogue, in the form all of the dense layer's
// products share:
//   Z[j][m] = sum_k A(m, k) B(j, k) + bias[m],  Out[j][m] = act(Z) + residual[j][m]
// (m is the output's contiguous index.) An operand is stored K-major (rows of
// k) or, with a_mn / b_mn, MN-major (rows of m or j).
//   forward: A = W, B = X;  dX: A = W (MN), B = dZ;  dW: A = X (MN), B = dZ (MN)
struct LinearGemm {
  const void* A = nullptr;
  const void* B = nullptr;
  bool a_mn = false, b_mn = false;
  int64_t M = 0, J = 0, K = 0;
  const void* bias = nullptr;
  const void* residual = nullptr;
  int act = DYRA_ACT_NONE;
  void* Out = nullptr;
  void* Z = nullptr;
  int* status = nullptr;
  float* ws = nullptr;      // tensor cores: linear_ws_bytes of scratch
  int* counters = nullptr;  // tensor cores: linear_counters ints, zero between calls
  // diagnostic limit of one pipeline wait of the clusters' kernel (0: the default)
  unsigned long long wait_ns = 0;
};

// CUDA-core products: fp32 (layers_f32.cu), and bf16 for DYRA_KERNELS=simt
// (layers_simt.cu).
int launch_linear_f32(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s);
int launch_linear_simt(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s);

// Tensor-core product of bf16 operands (layers_umma.cu).
int launch_linear_umma(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s);
size_t linear_ws_bytes(const DeviceInfo& dev);
int linear_counters(const DeviceInfo& dev);

// dZ = dY act'(Z) (skipped for DYRA_ACT_NONE) and its column sums (skipped
// when dbias is NULL). partial: kColSumChunks x d_out floats; counters:
// col_sum_blocks(d_out) ints, zero before and after the call.
constexpr int kColSumChunks = 64;
int col_sum_blocks(int d_out);
template <typename T>
int launch_act_backward(const T* dY, const T* Z, int act, T* dZ, T* dbias, int64_t N, int d_out,
                        float* partial, int* counters, int* status, const DeviceInfo& dev,
                        cudaStream_t s);

// ---- experts ----

constexpr int kMoeTokens = 64;  // tokens of one pass over the experts' weights

struct MoeShape {
  int d, f, experts, top_k, act, renorm;
};

// The router, kRouteTokens tokens per launch. logits: moe_logit_bytes of scratch;
// counters: moe_route_counters ints, zero before and after the call.
constexpr int kRouteTokens = 1024;
size_t moe_logit_bytes(const MoeShape& m);
int moe_route_counters();
template <typename T>
int launch_moe_route(const MoeShape& m, const T* X, const T* Wr, int* ids, float* weights,
                     int64_t N, double* logits, int* counters, cudaStream_t s);

// The experts' two products in fp32 (layers_f32.cu): hidden, then part.
int launch_moe_tiles_f32(const MoeShape& m, const float* X, const int* ids, const float* Wgu,
                         const float* Wd, int N, float* hidden, float* part, int* status,
                         const DeviceInfo& dev, cudaStream_t s);

// CUDA-core experts for N <= kMoeTokens tokens. hidden: N * top_k x f values,
// part: N * top_k x d floats.
template <typename T>
int launch_moe_experts_simt(const MoeShape& m, const T* X, const int* ids, const float* weights,
                            const T* Wgu, const T* Wd, const T* residual, T* Y, int N, T* hidden,
                            float* part, int* status, const DeviceInfo& dev, cudaStream_t s);

// Tensor-core experts for N <= kMoeTokens tokens (layers_moe_umma.cu). hidden:
// moe_reached_max x kMoeTokens x f values; ws and counters (zero between calls)
// as the sizes below.
int moe_reached_max(const MoeShape& m);
int moe_counters(const MoeShape& m);
size_t moe_ws_bytes(const MoeShape& m, const DeviceInfo& dev);
int launch_moe_experts_umma(const MoeShape& m, const __nv_bfloat16* X, const int* ids,
                            const float* weights, const __nv_bfloat16* Wgu,
                            const __nv_bfloat16* Wd, const __nv_bfloat16* residual,
                            __nv_bfloat16* Y, int N, __nv_bfloat16* hidden, float* ws,
                            int* counters, int* status, unsigned long long wait_ns,
                            const DeviceInfo& dev, cudaStream_t s);

}  // namespace dyra
