// layers_f32.cu - the fp32 products of the dense layer and of the experts on the
// CUDA cores: plain FFMA (TF32 tensor cores would lose ~1e-3).
//
// An Out tile of BT x BT on 256 threads of (BT/16)^2 values each, k in steps of 32
// through a ring of three shared-memory buffers filled by asynchronous copies.
// An operand's tile is kept as it is stored, rows of k (K-major) or rows of k over
// consecutive m (MN-major), so the copies are 16 bytes where the stored rows are
// 16-byte aligned and single values otherwise (odd sizes). Small products are
// bound by the latency of their few steps: a tile's steps are then shared by a
// cluster of cs CTAs, whose parts meet in distributed shared memory, in order.
#include <algorithm>

#include "layers.h"
#include "layers_math.cuh"
#include "sm100.cuh"

namespace dyra {

namespace {

using sm100::cluster_ctarank;
using sm100::cluster_sync_all;
using sm100::mapa_shared;
using sm100::smem_u32;

constexpr int kBk = 32, kRing = 3;

template <int BT>
struct F32Tile {
  static constexpr int V = BT / 16;                 // values per thread and side
  static constexpr int LdK = kBk + 4;               // K-major: [BT][LdK]
  static constexpr int LdM = BT + 4;                // MN-major: [kBk][LdM]
  static constexpr int Buf = BT * LdK > kBk * LdM ? BT * LdK : kBk * LdM;  // floats
  static constexpr int Part = BT * BT;
  static constexpr int Floats = 2 * kRing * Buf > Part ? 2 * kRing * Buf : Part;
};

// 4 bytes, or zero
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The BT x kBk tile at (r0, k0) of an operand of `rows` rows and K columns.
template <int BT, bool MN, bool VEC>
__device__ __forceinline__ void copy_tile(uint32_t dst, const float* __restrict__ src, int64_t rows,
                                          int64_t K, int64_t r0, int64_t k0) {
  using S = F32Tile<BT>;
  constexpr int W = VEC ? 4 : 1;  // values per copy
  constexpr int Count = BT * kBk / W;
#pragma unroll
  for (int i = 0; i < (Count + 255) / 256; ++i) {
    const int idx = threadIdx.x + 256 * i;
    if (Count % 256 && idx >= Count) break;
    int r, k;
    if (MN) {
      r = idx % (BT / W) * W;
      k = idx / (BT / W);
    } else {
      k = idx % (kBk / W) * W;
      r = idx / (kBk / W);
    }
    const int64_t gr = r0 + r, gk = k0 + k;
    const bool in = gr < rows && gk < K;
    const float* from = src + (in ? (MN ? gk * rows + gr : gr * K + gk) : 0);
    const uint32_t to = dst + 4u * static_cast<uint32_t>(MN ? k * S::LdM + r : r * S::LdK + k);
    if (VEC)
      sm100::cp_async_16(to, from, in ? 16u : 0u);
    else
      cp_async_4(to, from, in);
  }
}

// A thread's V rows of a side: t + 16 v of a K-major operand, 4 t + 64 (v / 4) + v % 4
// (V >= 4) or V t + v of an MN-major one.
template <int BT, bool MN>
__device__ __forceinline__ int side_row(int t, int v) {
  constexpr int V = F32Tile<BT>::V;
  if (!MN) return t + 16 * v;
  return V >= 4 ? 4 * t + 64 * (v / 4) + v % 4 : V * t + v;
}
// Two fp32 FMAs in one instruction on the halves of 64-bit registers, which halves
// the issue slots of the inner product (dW of 512 rows, 2048 -> 2048: 150 -> 109 us
// with 128 tiles; the forward, bound by its shared-memory loads, is as before).
__device__ __forceinline__ void add_product(f32x2& d, f32x2 a, f32x2 b) { d = fma2(a, b, d); }

// A's side of the product, four k of a buffer: acc(y, x) += sum over k of a b.
// K-major A (then B is K-major too): the halves are even and odd k, both operands
// as they lie; MN-major A: the halves are two neighbouring x, b goes to both.
template <int BT, bool AMN, bool BMN>
struct Product {
  using S = F32Tile<BT>;
  static constexpr int V = S::V, XN = AMN ? V / 2 : V;
  static_assert(AMN || !BMN, "a K-major A comes with a K-major B");
  f32x2 acc[V][XN];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int y = 0; y < V; ++y)
#pragma unroll
      for (int x = 0; x < XN; ++x) acc[y][x] = 0ull;
  }
  __device__ __forceinline__ void step(const float* as, const float* bs, int tx, int ty, int k) {
    if constexpr (!AMN) {
      ulonglong2 a[V], b[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        a[v] = *reinterpret_cast<const ulonglong2*>(as + (tx + 16 * v) * S::LdK + k);
        b[v] = *reinterpret_cast<const ulonglong2*>(bs + (ty + 16 * v) * S::LdK + k);
      }
#pragma unroll
      for (int y = 0; y < V; ++y)
#pragma unroll
        for (int x = 0; x < V; ++x) add_product(acc[y][x], a[x].x, b[y].x);
#pragma unroll
      for (int y = 0; y < V; ++y)
#pragma unroll
        for (int x = 0; x < V; ++x) add_product(acc[y][x], a[x].y, b[y].y);
    } else {
      float b[4][V];
      if constexpr (!BMN) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float4 q = *reinterpret_cast<const float4*>(bs + (ty + 16 * v) * S::LdK + k);
          b[0][v] = q.x, b[1][v] = q.y, b[2][v] = q.z, b[3][v] = q.w;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x2 a[XN];
        const float* row = as + (k + q) * S::LdM;
        if constexpr (V >= 4) {
#pragma unroll
          for (int g = 0; g < V / 4; ++g) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(row + 4 * tx + 64 * g);
            a[2 * g] = w.x, a[2 * g + 1] = w.y;
          }
        } else {
          a[0] = *reinterpret_cast<const f32x2*>(row + 2 * tx);
        }
        if constexpr (BMN) {
          const float* br = bs + (k + q) * S::LdM;
          if constexpr (V >= 4) {
#pragma unroll
            for (int g = 0; g < V / 4; ++g) {
              const float4 w = *reinterpret_cast<const float4*>(br + 4 * ty + 64 * g);
              b[q][4 * g] = w.x, b[q][4 * g + 1] = w.y, b[q][4 * g + 2] = w.z;
              b[q][4 * g + 3] = w.w;
            }
          } else {
#pragma unroll
            for (int v = 0; v < V; ++v) b[q][v] = br[V * ty + v];
          }
        }
#pragma unroll
        for (int y = 0; y < V; ++y) {
          const f32x2 by = pair(b[q][y], b[q][y]);
#pragma unroll
          for (int x = 0; x < XN; ++x) add_product(acc[y][x], a[x], by);
        }
      }
    }
  }
  __device__ __forceinline__ float value(int y, int x) const {
    if constexpr (AMN) {
      const float2 h = halves(acc[y][x / 2]);
      return x & 1 ? h.y : h.x;
    } else {
      const float2 h = halves(acc[y][x]);
      return h.x + h.y;
    }
  }
};

__device__ __forceinline__ void finish_f32(const LinearGemm& g, int64_t j, int64_t m, float z) {
  const size_t at = static_cast<size_t>(j) * g.M + m;
  if (!sm100::in_bounds(g.status, at, 1, static_cast<size_t>(g.J) * g.M)) return;
  if (g.bias) z += static_cast<const float*>(g.bias)[m];
  if (g.Z) static_cast<float*>(g.Z)[at] = z;
  float y = z;
  with_act(g.act, [&](auto tag) { y = act_f<decltype(tag)::value>(z); });
  if (g.residual) y += static_cast<const float*>(g.residual)[at];
  static_cast<float*>(g.Out)[at] = y;
}

template <int BT, bool AMN, bool BMN, bool VEC>
__global__ void __launch_bounds__(256)
    linear_f32_kernel(const __grid_constant__ LinearGemm g, int64_t m_tiles, int cs) {
  using S = F32Tile<BT>;
  constexpr int V = S::V;
  extern __shared__ __align__(16) float smem[];
  // the next grid is not let in early: its blocks, placed beside these as they
  // leave, would share the SMs unevenly (dX and dW of 240 rows, 1346 -> 760: 79 us
  // instead of 58)
  sm100::pdl_wait();
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t tile = blockIdx.x / cs;
  const int64_t jt = tile / m_tiles;
  const int64_t m0 = (tile - jt * m_tiles) * BT, j0 = jt * BT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float* A = static_cast<const float*>(g.A);
  const float* B = static_cast<const float*>(g.B);
  const int64_t steps = (g.K + kBk - 1) / kBk;
  const int64_t s0 = rank * steps / cs, s1 = (rank + 1) * steps / cs;
  const uint32_t base = smem_u32(smem);
  auto issue = [&](int64_t s) {
    if (s < s1) {
      const uint32_t at = base + static_cast<uint32_t>((s - s0) % kRing) * (2u * S::Buf * 4u);
      copy_tile<BT, AMN, VEC>(at, A, g.M, g.K, m0, s * kBk);
      copy_tile<BT, BMN, VEC>(at + S::Buf * 4u, B, g.J, g.K, j0, s * kBk);
    }
    sm100::cp_async_commit();  // one group per step, empty beyond the last
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(s0 + i);
  Product<BT, AMN, BMN> sum;
  sum.clear();
  for (int64_t s = s0; s < s1; ++s) {
    cp_async_wait<kRing - 2>();
    __syncthreads();  // step s has landed, and step s - 1's buffer is no longer read
    issue(s + kRing - 1);
    const float* as = smem + static_cast<size_t>((s - s0) % kRing) * 2 * S::Buf;
    const float* bs = as + S::Buf;
#pragma unroll
    for (int k = 0; k < kBk; k += 4) sum.step(as, bs, tx, ty, k);
  }
  if (cs == 1) {
#pragma unroll
    for (int y = 0; y < V; ++y) {
      const int64_t j = j0 + side_row<BT, BMN>(ty, y);
#pragma unroll
      for (int x = 0; x < V; ++x) {
        const int64_t m = m0 + side_row<BT, AMN>(tx, x);
        if (j < g.J && m < g.M) finish_f32(g, j, m, sum.value(y, x));
      }
    }
    return;
  }
  cp_async_wait<0>();
  __syncthreads();  // the buffers hold the part [BT][BT] now
#pragma unroll
  for (int y = 0; y < V; ++y)
#pragma unroll
    for (int x = 0; x < V; ++x)
      smem[side_row<BT, BMN>(ty, y) * BT + side_row<BT, AMN>(tx, x)] = sum.value(y, x);
  cluster_sync_all();
  const int r0 = rank * BT / cs, r1 = (rank + 1) * BT / cs;
  for (int i = r0 * BT + static_cast<int>(threadIdx.x); i < r1 * BT; i += 256) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = q < cs ? ld_shared_cluster(mapa_shared(base + 4u * i, static_cast<uint32_t>(q))) : 0.f;
    float z = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < cs) z += v[q];
    const int64_t j = j0 + i / BT, m = m0 + i % BT;
    if (j < g.J && m < g.M) finish_f32(g, j, m, z);
  }
  cluster_sync_all();  // no CTA leaves while its part is read
}

// ---------------------------------------------------------------- experts ----
// The experts in fp32: 64 weight rows of one expert per block against the slots
// (token, k) that name it, sixteen at a time, k in steps of 32 through a ring of
// four buffers. STAGE 0: rows f of the gate and of the up matrix together, hidden
// [slot] = act(g) u; STAGE 1: rows d, part[slot]. The weights are read once for
// every sixteen slots; 128 threads, 4 rows (of each matrix) x 2 slots each. A cluster
// of cs blocks shares the steps of a tile, as in the dense products.
constexpr int kExRows = 64, kExSlots = 16, kExRing = 4;

template <int STAGE>
struct ExpertTile {
  static constexpr int NG = STAGE == 0 ? 2 : 1;
  static constexpr int Ld = kBk + 4;
  static constexpr int Buf = (NG * kExRows + kExSlots) * Ld;
};

template <int STAGE, bool VEC>
__global__ void __launch_bounds__(128)
    moe_tile_kernel(MoeShape m, const float* __restrict__ In, const int* __restrict__ ids,
                    const float* __restrict__ W, float* __restrict__ Out, int N, int* status, int cs) {
  using S = ExpertTile<STAGE>;
  constexpr int NG = S::NG, Ld = S::Ld, W4 = VEC ? 4 : 1;
  extern __shared__ __align__(16) float smem[];
  __shared__ int list[kMoeTokens * DYRA_MOE_MAX_TOP_K];
  __shared__ int count;
  sm100::pdl_wait();
  const int e = blockIdx.y, tid = threadIdx.x;
  const int slots = N * m.top_k;
  if (tid < 32) {  // the expert's slots, in order
    int c = 0;
    for (int i0 = 0; i0 < slots; i0 += 32) {
      const int i = i0 + tid;
      const bool hit = i < slots && ids[i] == e;
      const unsigned b = __ballot_sync(0xffffffffu, hit);
      if (hit) list[c + __popc(b & ((1u << tid) - 1))] = i;
      c += __popc(b);
    }
    if (tid == 0) count = c;
  }
  __syncthreads();
  const int nsl = count;
  if (nsl == 0) return;
  const int rows = STAGE == 0 ? m.f : m.d, K = STAGE == 0 ? m.d : m.f;
  const size_t wrows = STAGE == 0 ? 2 * static_cast<size_t>(m.f) : m.d;
  const float* We = W + wrows * e * K;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int r0 = static_cast<int>(blockIdx.x) / cs * kExRows;
  const int tx = tid & 15, ty = tid >> 4;
  const int all = (K + kBk - 1) / kBk;
  const int first = rank * all / cs, steps = (rank + 1) * all / cs - first;
  const uint32_t base = smem_u32(smem);
  const size_t extent = static_cast<size_t>(slots) * rows;
  for (int s0 = 0; s0 < nsl; s0 += kExSlots) {
    auto issue = [&](int s) {
      if (s < steps) {
        const uint32_t at = base + static_cast<uint32_t>(s % kExRing) * (S::Buf * 4u);
        const int k0 = (first + s) * kBk;
#pragma unroll
        for (int i = 0; i < (NG * kExRows + kExSlots) * kBk / W4 / 128; ++i) {
          const int idx = tid + 128 * i;
          const int k = idx % (kBk / W4) * W4, r = idx / (kBk / W4);
          const float* row;
          bool in = k0 + k < K;
          if (r < NG * kExRows) {
            const int wr = r0 + r % kExRows;
            in = in && wr < rows;
            row = We + static_cast<size_t>(r < kExRows ? wr : m.f + wr) * K;
          } else {
            const int sl = s0 + r - NG * kExRows;
            in = in && sl < nsl;
            const int slot = list[in ? sl : 0];
            row = In + static_cast<size_t>(STAGE == 0 ? slot / m.top_k : slot) * K;
          }
          const uint32_t to = at + 4u * static_cast<uint32_t>(r * Ld + k);
          const float* from = in ? row + k0 + k : In;
          if (VEC)
            sm100::cp_async_16(to, from, in ? 16u : 0u);
          else
            cp_async_4(to, from, in);
        }
      }
      sm100::cp_async_commit();
    };
    f32x2 acc[NG][4][2] = {};
#pragma unroll
    for (int i = 0; i < kExRing - 1; ++i) issue(i);
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<kExRing - 2>();
      __syncthreads();
      issue(s + kExRing - 1);
      const float* buf = smem + static_cast<size_t>(s % kExRing) * S::Buf;
      const float* xs = buf + NG * kExRows * Ld;
#pragma unroll
      for (int k = 0; k < kBk; k += 4) {
        ulonglong2 x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          x[j] = *reinterpret_cast<const ulonglong2*>(xs + (ty + 8 * j) * Ld + k);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(
                buf + (g * kExRows + tx + 16 * i) * Ld + k);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              add_product(acc[g][i][j], w.x, x[j].x);
              add_product(acc[g][i][j], w.y, x[j].y);
            }
          }
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // the ring is free
    auto out = [&](int sl, int r, float v, float u) {
      const int row = r0 + r;
      if (sl >= nsl || row >= rows) return;
      const size_t at = static_cast<size_t>(list[sl]) * rows + row;
      if (!sm100::in_bounds(status, at, 1, extent)) return;
      if (STAGE == 0)
        with_act(m.act, [&](auto tag) { v = act_f<decltype(tag)::value>(v) * u; });
      Out[at] = v;
    };
    if (cs == 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = halves(acc[0][i][j]), u = halves(acc[NG - 1][i][j]);
          out(s0 + ty + 8 * j, tx + 16 * i, a.x + a.y, u.x + u.y);
        }
      continue;
    }
    // the part [slot][matrix][row], then a share of the values summed over the parts
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = halves(acc[g][i][j]);
          smem[((ty + 8 * j) * NG + g) * kExRows + tx + 16 * i] = a.x + a.y;
        }
    cluster_sync_all();
    constexpr int Values = kExSlots * kExRows;
    for (int i = rank * Values / cs + tid; i < (rank + 1) * Values / cs; i += 128) {
      const int sl = i / kExRows, r = i % kExRows;
      float v = 0.f, u = 0.f;
      for (int q = 0; q < cs; ++q) {
        const uint32_t at = mapa_shared(base + 4u * static_cast<uint32_t>(sl * NG * kExRows + r),
                                        static_cast<uint32_t>(q));
        v += ld_shared_cluster(at);
        if (STAGE == 0) u += ld_shared_cluster(at + 4u * kExRows);
      }
      out(s0 + sl, r, v, u);
    }
    cluster_sync_all();  // the parts have been read: the ring may start again
  }
}

template <int STAGE, bool VEC>
int launch_experts(const MoeShape& m, const float* In, const int* ids, const float* W, float* Out,
                   int N, int* status, const DeviceInfo& dev, cudaStream_t s) {
  auto kfn = moe_tile_kernel<STAGE, VEC>;
  static KernelSetup setup;
  constexpr uint32_t smem = kExRing * ExpertTile<STAGE>::Buf * 4;
  if (raise_smem(kfn, setup, dev.device, smem, false)) return -1;
  const int rows = STAGE == 0 ? m.f : m.d, steps = ((STAGE == 0 ? m.d : m.f) + kBk - 1) / kBk;
  const int tiles = (rows + kExRows - 1) / kExRows, reached = std::min(m.experts, N * m.top_k);
  // clusters while the blocks are fewer than two per SM and each keeps four steps
  int cs = 1;
  while (cs < 8 && tiles * reached * cs < 2 * dev.sm_count && 8 * cs <= steps) cs *= 2;
  return launch_dependent(kfn, dim3(tiles * cs, m.experts), dim3(128), smem, cs, s, m, In, ids, W,
                          Out, N, status, cs);
}

template <int BT, bool AMN, bool BMN, bool VEC>
int launch_tile(const LinearGemm& g, int cs, const DeviceInfo& dev, cudaStream_t s) {
  auto kfn = linear_f32_kernel<BT, AMN, BMN, VEC>;
  static KernelSetup setup;
  constexpr uint32_t smem = F32Tile<BT>::Floats * 4;
  if (raise_smem(kfn, setup, dev.device, smem, false)) return -1;
  const int64_t mt = (g.M + BT - 1) / BT, jt = (g.J + BT - 1) / BT;
  if (mt * jt * cs > 0x7fffffffll) return -1;
  return launch_dependent(kfn, dim3(static_cast<unsigned>(mt * jt * cs)), dim3(256), smem, cs, s, g,
                          mt, cs);
}

template <int BT>
int launch_bt(const LinearGemm& g, int cs, const DeviceInfo& dev, cudaStream_t s) {
  // 16-byte copies need every stored row to start on 16 bytes
  const int64_t la = g.a_mn ? g.M : g.K, lb = g.b_mn ? g.J : g.K;
  const bool vec = la % 4 == 0 && lb % 4 == 0;
  if (g.a_mn && g.b_mn)
    return vec ? launch_tile<BT, true, true, true>(g, cs, dev, s)
               : launch_tile<BT, true, true, false>(g, cs, dev, s);
  if (g.a_mn)
    return vec ? launch_tile<BT, true, false, true>(g, cs, dev, s)
               : launch_tile<BT, true, false, false>(g, cs, dev, s);
  return vec ? launch_tile<BT, false, false, true>(g, cs, dev, s)
             : launch_tile<BT, false, false, false>(g, cs, dev, s);
}

}  // namespace

// Tile and cluster by a model in microseconds, fitted to 64 x 256 -> 256 up to
// 1024 x 1024 -> 1024 and 512 x 2048 -> 2048: a step of a 128, 64 or 32 tile takes
// its SM about 3.9, 1.25 or 0.5, and joining a cluster's parts 6, 1.5 or 0.7 (512 x
// 512 -> 512: 14.8 with 64 tiles in clusters of 4, 25.6 alone, 24.3 with 128 tiles).
int launch_linear_f32(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t steps = (g.K + kBk - 1) / kBk;
  int best_bt = 128, best_cs = 1;
  double best = -1.0;
  for (int bt : {128, 64, 32}) {
    const int64_t tiles = ((g.M + bt - 1) / bt) * ((g.J + bt - 1) / bt);
    const double step = bt == 128 ? 3.9 : bt == 64 ? 1.25 : 0.5;
    const double join = bt == 128 ? 6.0 : bt == 64 ? 1.5 : 0.7;
    for (int cs = 1; cs <= 8 && cs <= steps; cs *= 2) {
      if (cs > 1 && tiles * cs > 2 * dev.sm_count) break;
      const double rounds = static_cast<double>((tiles * cs + dev.sm_count - 1) / dev.sm_count);
      const double us = rounds * step * static_cast<double>((steps + cs - 1) / cs) +
                        (cs > 1 ? join : 0.0);
      if (best < 0.0 || us < best) {
        best = us;
        best_bt = bt;
        best_cs = cs;
      }
    }
  }
  if (best_bt == 128) return launch_bt<128>(g, best_cs, dev, s);
  if (best_bt == 64) return launch_bt<64>(g, best_cs, dev, s);
  return launch_bt<32>(g, best_cs, dev, s);
}

int launch_moe_tiles_f32(const MoeShape& m, const float* X, const int* ids, const float* Wgu,
                         const float* Wd, int N, float* hidden, float* part, int* status,
                         const DeviceInfo& dev, cudaStream_t s) {
  // a stage's rows are whole 16-byte pieces: of d values in the first, f in the second
  if (m.d % 4 ? launch_experts<0, false>(m, X, ids, Wgu, hidden, N, status, dev, s)
              : launch_experts<0, true>(m, X, ids, Wgu, hidden, N, status, dev, s))
    return -1;
  return m.f % 4 ? launch_experts<1, false>(m, hidden, ids, Wd, part, N, status, dev, s)
                 : launch_experts<1, true>(m, hidden, ids, Wd, part, N, status, dev, s);
}

}  // namespace dyra
