// layers_simt.cu - CUDA-core kernels of the dense and expert layers: the
// activation's backward with its column sums, the router, the experts of fp32
// handles, and the debugging variant of the bf16 products.
#include <algorithm>

#include "layers.h"
#include "layers_math.cuh"
#include "sm100.cuh"

namespace dyra {

namespace {

// ------------------------------------------------------- bf16 dense gemm ----
// The debugging variant of the bf16 products: 64 x 64 of Out per block of 256
// threads, k in steps of 16 through shared memory in fp32.
constexpr int kSimtBt = 64, kSimtBk = 16;

template <bool AMN, bool BMN>
__global__ void __launch_bounds__(256) linear_simt_kernel(LinearGemm g, int64_t m_tiles) {
  using T = __nv_bfloat16;
  __shared__ float As[kSimtBk][kSimtBt + 1];
  __shared__ float Bs[kSimtBk][kSimtBt + 1];
  const T* __restrict__ A = static_cast<const T*>(g.A);
  const T* __restrict__ B = static_cast<const T*>(g.B);
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t jt = blockIdx.x / m_tiles;
  const int64_t m0 = (blockIdx.x - jt * m_tiles) * kSimtBt, j0 = jt * kSimtBt;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < g.K; k0 += kSimtBk) {
    for (int idx = threadIdx.x; idx < kSimtBt * kSimtBk; idx += 256) {
      const int ka = AMN ? idx / kSimtBt : idx % kSimtBk, ma = AMN ? idx % kSimtBt : idx / kSimtBk;
      const int kb = BMN ? idx / kSimtBt : idx % kSimtBk, jb = BMN ? idx % kSimtBt : idx / kSimtBk;
      const int64_t gm = m0 + ma, gka = k0 + ka, gj = j0 + jb, gkb = k0 + kb;
      As[ka][ma] = gm < g.M && gka < g.K ? load_f(A[AMN ? gka * g.M + gm : gm * g.K + gka]) : 0.f;
      Bs[kb][jb] = gj < g.J && gkb < g.K ? load_f(B[BMN ? gkb * g.J + gj : gj * g.K + gkb]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSimtBk; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[j][m] = fmaf(Bs[k][ty + 16 * j], As[k][tx + 16 * m], acc[j][m]);
    __syncthreads();
  }
  const T* __restrict__ bias = static_cast<const T*>(g.bias);
  const T* residual = static_cast<const T*>(g.residual);  // may be Out: no __restrict__
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t gj = j0 + ty + 16 * j;
    if (gj >= g.J) continue;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t gm = m0 + tx + 16 * m;
      if (gm >= g.M) continue;
      const size_t at = static_cast<size_t>(gj) * g.M + gm;
      if (!sm100::in_bounds(g.status, at, 1, static_cast<size_t>(g.J) * g.M)) continue;
      float z = acc[j][m];
      if (bias) z += load_f(bias[gm]);
      if (g.Z) static_cast<T*>(g.Z)[at] = store_f<T>(z);
      with_act(g.act, [&](auto tag) { z = act_f<decltype(tag)::value, true>(z); });
      if (residual) z += load_f(residual[at]);
      static_cast<T*>(g.Out)[at] = store_f<T>(z);
    }
  }
}

// ---------------------------------------------------- activation backward ----
// dZ = dY act'(Z) and the column sums of dZ, in one pass over dY and Z. A block
// takes 32 V columns (V values per thread: one 16-byte piece where rows are
// aligned, else single values) and every 8 x chunks-th row; the sums of its 8
// row lanes meet in shared memory, the chunks' sums in `partial`, and the last
// block of a column group to arrive adds the chunks in order and rounds once.
// The pass is bound by the bytes it has in flight: four rows per thread, and as many
// blocks as are resident at once: two per SM with Z, four without. 6432 x 4096 values
// with the GELU take 35.3 us (4.5 TB/s; the ReLU 28.4, 5.6 TB/s), the column sums alone
// 13.8. When this was chosen, with a GELU of 32.8: four blocks per SM 35.5, three rows
// per thread 32.5 to 49.8 (GELU) and 42 (ReLU), the GELU's slope one value at a time
// 33.4; the sums alone 12.4, with two blocks per SM 14.6.
template <int ACT>
constexpr int kActBlocks = ACT == DYRA_ACT_NONE ? 4 : 2;

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(256, kActBlocks<ACT>)
    act_backward_kernel(const T* dY, const T* Z, T* dZ, T* __restrict__ dbias, int64_t N, int d_out,
                        float* __restrict__ partial, int* counters, int* status) {
  struct alignas(sizeof(T) * V) P {
    T v[V];
  };
  if (sizeof(T) == 2) sm100::pdl_launch_dependents();  // not before the fp32 products: layers_f32.cu
  sm100::pdl_wait();
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int col = (blockIdx.x * 32 + lane) * V;
  float sum[V] = {};
  if (col < d_out) {
    constexpr int kRows = 4;  // rows of a thread in flight
    const int64_t stride = static_cast<int64_t>(gridDim.y) * 8;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 8 + rl; r0 < N; r0 += kRows * stride) {
      P g[kRows], z[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t r = r0 + u * stride;
        const size_t at = static_cast<size_t>(r) * d_out + col;
        if (r < N && sm100::in_bounds(status, at, V, static_cast<size_t>(N) * d_out)) {
          g[u] = *reinterpret_cast<const P*>(dY + at);
          if (ACT != DYRA_ACT_NONE) z[u] = *reinterpret_cast<const P*>(Z + at);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t r = r0 + u * stride;
        const size_t at = static_cast<size_t>(r) * d_out + col;
        if (r >= N || !sm100::in_bounds(status, at, V, static_cast<size_t>(N) * d_out)) continue;
        P out;
        float slope[V];
        if constexpr (ACT != DYRA_ACT_NONE) {
#pragma unroll
          for (int i = 0; i < V; ++i) slope[i] = load_f(z[u].v[i]);
          if constexpr (V == 8) {
            act_grad8<ACT>(slope);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) slope[i] = act_grad_f<ACT>(slope[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float d = load_f(g[u].v[i]);
          // a zero slope of the ReLU is a zero gradient, whatever dY holds
          if (ACT == DYRA_ACT_RELU)
            d = slope[i] > 0.f ? d : 0.f;
          else if (ACT != DYRA_ACT_NONE)
            d *= slope[i];
          sum[i] += d;
          // bf16: the tensor cores' operand of both products, rounded once (the sums
          // are not); the gradients' error goes from 0.0017 to 0.0024
          out.v[i] = store_f<T>(d);
        }
        if (ACT != DYRA_ACT_NONE) *reinterpret_cast<P*>(dZ + at) = out;
      }
    }
  }
  if (dbias == nullptr) return;
  __shared__ float red[8][32 * V + 1];
  __shared__ int last;
#pragma unroll
  for (int i = 0; i < V; ++i) red[rl][lane * V + i] = sum[i];
  __syncthreads();
  const int c0 = blockIdx.x * 32 * V;
  for (int c = threadIdx.x; c < 32 * V; c += 256) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += red[q][c];
    if (c0 + c < d_out) partial[static_cast<size_t>(blockIdx.y) * d_out + c0 + c] = t;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(&counters[blockIdx.x], 1) == static_cast<int>(gridDim.y) - 1;
    if (last) counters[blockIdx.x] = 0;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int c = threadIdx.x; c < 32 * V; c += 256) {
    if (c0 + c >= d_out) continue;
    float t = 0.f;
    for (int q = 0; q < static_cast<int>(gridDim.y); ++q)
      t += __ldcg(partial + static_cast<size_t>(q) * d_out + c0 + c);
    dbias[c0 + c] = store_f<T>(t);
  }
}

template <typename T, int V>
int launch_act_backward_v(const T* dY, const T* Z, int act, T* dZ, T* dbias, int64_t N, int d_out,
                          float* partial, int* counters, int* status, const DeviceInfo& dev,
                          cudaStream_t s) {
  const int cols = (d_out + 32 * V - 1) / (32 * V);
  // every block with at least one row per lane
  const int per_sm = act == DYRA_ACT_NONE ? kActBlocks<DYRA_ACT_NONE> : kActBlocks<DYRA_ACT_RELU>;
  const int64_t want = std::max<int64_t>(1, per_sm * dev.sm_count / cols);
  const int chunks = static_cast<int>(
      std::min<int64_t>({want, std::max<int64_t>(1, (N + 7) / 8), kColSumChunks}));
  int rc = -1;
  with_act_host(act, [&](auto tag) {
    rc = launch_dependent(act_backward_kernel<T, V, decltype(tag)::value>, dim3(cols, chunks),
                          dim3(256), 0, 1, s, dY, Z, dZ, dbias, N, d_out, partial, counters, status);
  });
  return rc;
}

// ----------------------------------------------------------------- router ----
// Logits of four experts x four tokens per block, its 256 threads sharing d in
// pieces of eight. The choice of experts is discrete, so the sums are fp64, in
// which the products are exact: logits next to the border of the top k are told
// apart down to d 2^-53 of their products' size. The last block of a token group
// to arrive then picks, a warp per token, the largest logit top_k times.
constexpr int kRouteTile = 4;

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* __restrict__ row, int i, int d, float (&v)[8]) {
  if (VEC) {
    if (sizeof(T) == 2) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + i));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + i) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < d ? load_f(row[i + j]) : 0.f;
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
    moe_route_kernel(MoeShape m, const T* __restrict__ X, const T* __restrict__ Wr,
                     int* __restrict__ ids, float* __restrict__ weights,
                     double* __restrict__ logits, int* counters, int N) {
  constexpr int R = kRouteTile;
  __shared__ double red[8][R * R];
  __shared__ double pick[R][DYRA_MOE_MAX_EXPERTS];
  __shared__ int last;
  sm100::pdl_launch_dependents();  // the experts' kernel may set up meanwhile
  sm100::pdl_wait();
  const int e0 = blockIdx.x * R, n0 = blockIdx.y * R;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double acc[R][R] = {};
  for (int i = threadIdx.x * 8; i < m.d; i += 256 * 8) {
    float w[R][8], x[R][8];
#pragma unroll
    for (int q = 0; q < R; ++q) {  // beyond the last expert or token: the last, unused
      load8<T, VEC>(Wr + static_cast<size_t>(min(e0 + q, m.experts - 1)) * m.d, i, m.d, w[q]);
      load8<T, VEC>(X + static_cast<size_t>(min(n0 + q, N - 1)) * m.d, i, m.d, x[q]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double wd[R];
#pragma unroll
      for (int b = 0; b < R; ++b) wd[b] = w[b][j];
#pragma unroll
      for (int a = 0; a < R; ++a) {
        const double xd = x[a][j];
#pragma unroll
        for (int b = 0; b < R; ++b) acc[a][b] = fma(xd, wd[b], acc[a][b]);
      }
    }
  }
  // the sixteen sums over the warp: at each step a lane keeps half of its values
  // and hands the other half to its partner, so lane l ends with value l / 2
  double v[R * R];
#pragma unroll
  for (int a = 0; a < R; ++a)
#pragma unroll
    for (int b = 0; b < R; ++b) v[a * R + b] = acc[a][b];
#pragma unroll
  for (int o = 16, n = R * R / 2; n > 0; o >>= 1, n >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const double give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
  if ((lane & 1) == 0) red[warp][lane >> 1] = v[0];
  __syncthreads();
  if (threadIdx.x < R * R) {
    double t = 0.0;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += red[q][threadIdx.x];
    const int n = n0 + threadIdx.x / R, e = e0 + threadIdx.x % R;
    if (n < N && e < m.experts) logits[static_cast<size_t>(n) * m.experts + e] = t;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(&counters[blockIdx.y], 1) == static_cast<int>(gridDim.x) - 1;
    if (last) counters[blockIdx.y] = 0;
  }
  __syncthreads();
  const int n = n0 + warp;
  if (!last || warp >= R || n >= N) return;
  __threadfence();
  double* logit = pick[warp];
  for (int e = lane; e < m.experts; e += 32)
    logit[e] = __ldcg(logits + static_cast<size_t>(n) * m.experts + e);
  __syncwarp();
  // expert 32 i + lane is this lane's i-th; a set bit of taken marks a chosen one
  unsigned taken = 0;
  double top = 0.0;
  float mine = 0.f, sum = 0.f;
  int my_id = 0;
  const double ninf = -INFINITY;
  for (int k = 0; k < m.top_k; ++k) {
    double best = 0.0;
    int at = 0x7fffffff;
    for (int e = lane, i = 0; e < m.experts; e += 32, ++i) {
      if (taken >> i & 1) continue;
      const double v = isnan(logit[e]) ? ninf : logit[e];
      if (at == 0x7fffffff || v > best) best = v, at = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (oa != 0x7fffffff && (at == 0x7fffffff || ob > best || (ob == best && oa < at)))
        best = ob, at = oa;
    }
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    if (k == 0) top = logit[at];
    const float p = expf(static_cast<float>(logit[at] - top));
    sum += p;
    if (lane == k) mine = p, my_id = at;
  }
  if (!m.renorm) {
    sum = 0.f;
    for (int e = lane; e < m.experts; e += 32) sum += expf(static_cast<float>(logit[e] - top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (lane < m.top_k) {
    ids[static_cast<size_t>(n) * m.top_k + lane] = my_id;
    weights[static_cast<size_t>(n) * m.top_k + lane] = mine / sum;
  }
}

// ---------------------------------------------------------------- experts ----
// CUDA-core experts (fp32 with few slots per expert, and bf16 for debugging): a warp
// per output row of one expert, over the slots (token, k) that name it, up to eight at
// a time: each weight is read once per eight slots. STAGE 0: hidden[slot] = act(g) u
// over rows f; STAGE 1: part[slot] over rows d. The slots of the block's expert are
// listed in order first. VEC: the stage's rows are whole 16-byte pieces. A warp's time is the
// latency of its loads; two rows per warp, for half the loads of x, were slower (151
// against 94 us for 14 tokens on 5 experts of 601 x 1935).

// The sums over the warp of n values each lane holds: at each step a lane keeps half
// of its values and hands the other half to its partner, so lane l ends with value
// l / (32 / n) (n a power of two, at most 32).
template <int n>
__device__ __forceinline__ float sums_to_lanes(float (&v)[n], int lane) {
  int o = 16;
#pragma unroll
  for (int h = n / 2; h > 0; h >>= 1, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = upper ? v[i] : v[i + h], keep = upper ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (int q = 32 / n / 2; q > 0; q >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], q);
  return v[0];
}

template <typename T, int STAGE, bool VEC, int NS>
__device__ __forceinline__ void expert_row(const MoeShape& m, const T* __restrict__ In,
                                            const T* __restrict__ We, const int* list, int K,
                                            int rows, int row, int lane, T* __restrict__ hidden,
                                            float* __restrict__ part, size_t extent, int* status) {
  constexpr int W = VEC ? 16 / sizeof(T) : 1, NG = STAGE == 0 ? 2 : 1;
  struct alignas(W * sizeof(T)) P {
    T v[W];
  };
  const T* x[NS];
  const T* w[NG];
  float a[NG * NS] = {};
#pragma unroll
  for (int q = 0; q < NS; ++q)
    x[q] = In + static_cast<size_t>(STAGE == 0 ? list[q] / m.top_k : list[q]) * K;
#pragma unroll
  for (int g = 0; g < NG; ++g) w[g] = We + static_cast<size_t>(g * m.f + row) * K;
#pragma unroll 4
  for (int i = lane * W; i < K; i += 32 * W) {
    P pw[NG], px[NS];
#pragma unroll
    for (int g = 0; g < NG; ++g) pw[g] = *reinterpret_cast<const P*>(w[g] + i);
#pragma unroll
    for (int q = 0; q < NS; ++q) px[q] = *reinterpret_cast<const P*>(x[q] + i);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int j = 0; j < W; ++j)
          a[g * NS + q] = fmaf(load_f(pw[g].v[j]), load_f(px[q].v[j]), a[g * NS + q]);
  }
  constexpr int n = NG * NS, share = 32 / n;  // lanes per value
  const float v = sums_to_lanes<n>(a, lane);
  const float up = STAGE == 0 ? __shfl_xor_sync(0xffffffffu, v, 16) : 0.f;
  const int q = lane / share;
  if (lane % share != 0 || q >= NS) return;
  const size_t at = static_cast<size_t>(list[q]) * rows + row;
  if (!sm100::in_bounds(status, at, 1, extent)) return;
  if (STAGE == 0)
    with_act(m.act, [&](auto tag) {
      hidden[at] = store_f<T>(act_f<decltype(tag)::value, kFastMath<T>>(v) * up);
    });
  else
    part[at] = v;
}

template <typename T, int STAGE, bool VEC>
__global__ void __launch_bounds__(256)
    moe_expert_kernel(MoeShape m, const T* __restrict__ In, const int* __restrict__ ids,
                      const T* __restrict__ W, T* __restrict__ hidden, float* __restrict__ part,
                      int N, int* status) {
  __shared__ int list[kMoeTokens * DYRA_MOE_MAX_TOP_K];
  __shared__ int count;
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int e = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = N * m.top_k;
  if (warp == 0) {
    int c = 0;
    for (int i0 = 0; i0 < slots; i0 += 32) {
      const int i = i0 + lane;
      const bool hit = i < slots && ids[i] == e;
      const unsigned b = __ballot_sync(0xffffffffu, hit);
      if (hit) list[c + __popc(b & ((1u << lane) - 1))] = i;
      c += __popc(b);
    }
    if (lane == 0) count = c;
  }
  __syncthreads();
  const int nsl = count;
  const int rows = STAGE == 0 ? m.f : m.d, K = STAGE == 0 ? m.d : m.f;
  const size_t wrows = STAGE == 0 ? 2 * static_cast<size_t>(m.f) : m.d;
  const T* We = W + wrows * e * K;
  const size_t extent = static_cast<size_t>(slots) * rows;
  const int row = blockIdx.x * 8 + warp;
  if (row >= rows) return;
  int s0 = 0;
  auto take = [&](auto tag) {
    constexpr int NS = decltype(tag)::value;
    for (; s0 + NS <= nsl; s0 += NS)
      expert_row<T, STAGE, VEC, NS>(m, In, We, list + s0, K, rows, row, lane, hidden, part, extent,
                                    status);
  };
  take(ActTag<8>());
  take(ActTag<4>());
  take(ActTag<2>());
  take(ActTag<1>());
}

// Y[n] = sum over k, in order, of weights[n][k] part[n][k] + residual[n]
template <typename T>
__global__ void __launch_bounds__(256)
    moe_combine_kernel(MoeShape m, const int* __restrict__ ids, const float* __restrict__ weights,
                       const float* __restrict__ part, const T* residual, T* Y, int N,
                       int* status) {
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int n = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x;
  if (i >= m.d) return;
  float acc = 0.f;
  for (int k = 0; k < m.top_k; ++k) {
    const int slot = n * m.top_k + k, e = ids[slot];
    if (e >= 0 && e < m.experts)
      acc = fmaf(weights[slot], part[static_cast<size_t>(slot) * m.d + i], acc);
  }
  const size_t at = static_cast<size_t>(n) * m.d + i;
  if (!sm100::in_bounds(status, at, 1, static_cast<size_t>(N) * m.d)) return;
  if (residual) acc += load_f(residual[at]);
  Y[at] = store_f<T>(acc);
}

}  // namespace

int launch_linear_simt(const LinearGemm& g, const DeviceInfo&, cudaStream_t s) {
  const int64_t mt = (g.M + kSimtBt - 1) / kSimtBt, jt = (g.J + kSimtBt - 1) / kSimtBt;
  if (mt * jt > 0x7fffffffll) return -1;
  auto kfn = g.a_mn && g.b_mn ? linear_simt_kernel<true, true>
             : g.a_mn         ? linear_simt_kernel<true, false>
                              : linear_simt_kernel<false, false>;
  return launch_dependent(kfn, dim3(static_cast<unsigned>(mt * jt)), dim3(256), 0, 1, s, g, mt);
}

int col_sum_blocks(int d_out) { return (d_out + 31) / 32; }

template <typename T>
int launch_act_backward(const T* dY, const T* Z, int act, T* dZ, T* dbias, int64_t N, int d_out,
                        float* partial, int* counters, int* status, const DeviceInfo& dev,
                        cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if constexpr (sizeof(T) == 4)  // (bf16 rows are whole 16-byte pieces)
    if (d_out % V)
      return launch_act_backward_v<T, 1>(dY, Z, act, dZ, dbias, N, d_out, partial, counters, status,
                                         dev, s);
  return launch_act_backward_v<T, V>(dY, Z, act, dZ, dbias, N, d_out, partial, counters, status,
                                     dev, s);
}
template int launch_act_backward<float>(const float*, const float*, int, float*, float*, int64_t,
                                        int, float*, int*, int*, const DeviceInfo&, cudaStream_t);
template int launch_act_backward<__nv_bfloat16>(const __nv_bfloat16*, const __nv_bfloat16*, int,
                                                __nv_bfloat16*, __nv_bfloat16*, int64_t, int,
                                                float*, int*, int*, const DeviceInfo&,
                                                cudaStream_t);

size_t moe_logit_bytes(const MoeShape& m) {
  return static_cast<size_t>(kRouteTokens) * m.experts * sizeof(double);
}
int moe_route_counters() { return kRouteTokens / kRouteTile; }

template <typename T>
int launch_moe_route(const MoeShape& m, const T* X, const T* Wr, int* ids, float* weights,
                     int64_t N, double* logits, int* counters, cudaStream_t s) {
  const bool vec = m.d % 8 == 0;  // pieces of eight are whole and 16-byte aligned
  for (int64_t n0 = 0; n0 < N; n0 += kRouteTokens) {
    const int n = static_cast<int>(std::min<int64_t>(kRouteTokens, N - n0));
    const dim3 grid((m.experts + kRouteTile - 1) / kRouteTile, (n + kRouteTile - 1) / kRouteTile);
    auto kfn = vec ? moe_route_kernel<T, true> : moe_route_kernel<T, false>;
    if (launch_dependent(kfn, grid, dim3(256), 0, 1, s, m, X + n0 * m.d, Wr, ids + n0 * m.top_k,
                         weights + n0 * m.top_k, logits, counters, n))
      return -1;
  }
  return 0;
}
template int launch_moe_route<float>(const MoeShape&, const float*, const float*, int*, float*,
                                     int64_t, double*, int*, cudaStream_t);
template int launch_moe_route<__nv_bfloat16>(const MoeShape&, const __nv_bfloat16*,
                                             const __nv_bfloat16*, int*, float*, int64_t, double*,
                                             int*, cudaStream_t);

template <typename T>
int launch_moe_experts_simt(const MoeShape& m, const T* X, const int* ids, const float* weights,
                            const T* Wgu, const T* Wd, const T* residual, T* Y, int N, T* hidden,
                            float* part, int* status, const DeviceInfo& dev, cudaStream_t s) {
  bool tiles = false;
  if constexpr (sizeof(T) == 4) {
    // tiles of sixteen slots where the experts have about as many each: 280 slots on
    // 19 experts of 247 x 4961 take 278 us in tiles and took 742 by rows, 60 slots on 7
    // of 603 x 180 take 32 and 26
    tiles = N * m.top_k >= 12 * m.experts;
    if (tiles && launch_moe_tiles_f32(m, X, ids, Wgu, Wd, N, hidden, part, status, dev, s)) return -1;
  }
  if (!tiles) {
    // a stage's rows are whole 16-byte pieces: of d values in the first, f in the second
    auto up = m.d * sizeof(T) % 16 ? moe_expert_kernel<T, 0, false> : moe_expert_kernel<T, 0, true>;
    auto down = m.f * sizeof(T) % 16 ? moe_expert_kernel<T, 1, false> : moe_expert_kernel<T, 1, true>;
    if (launch_dependent(up, dim3((m.f + 7) / 8, m.experts), dim3(256), 0, 1, s, m, X, ids, Wgu,
                         hidden, static_cast<float*>(nullptr), N, status) ||
        launch_dependent(down, dim3((m.d + 7) / 8, m.experts), dim3(256), 0, 1, s, m,
                         static_cast<const T*>(hidden), ids, Wd, static_cast<T*>(nullptr), part, N,
                         status))
      return -1;
  }
  return launch_dependent(moe_combine_kernel<T>, dim3((m.d + 255) / 256, N), dim3(256), 0, 1, s, m,
                          ids, weights, static_cast<const float*>(part), residual, Y, N, status);
}
template int launch_moe_experts_simt<float>(const MoeShape&, const float*, const int*,
                                            const float*, const float*, const float*, const float*,
                                            float*, int, float*, float*, int*, const DeviceInfo&,
                                            cudaStream_t);
template int launch_moe_experts_simt<__nv_bfloat16>(
    const MoeShape&, const __nv_bfloat16*, const int*, const float*, const __nv_bfloat16*,
    const __nv_bfloat16*, const __nv_bfloat16*, __nv_bfloat16*, int, __nv_bfloat16*, float*, int*,
    const DeviceInfo&, cudaStream_t);

}  // namespace dyra
