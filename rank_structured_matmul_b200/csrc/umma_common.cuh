// umma_common.cuh - what the tensor-core files share on top of the GEMM
// skeletons: K-major descriptors, the bf16 store boxes of the epilogues, and the
// host side of a launch.
#pragma once

#include <algorithm>

#include "internal.h"
#include "umma_gemm.cuh"
#include "umma_gemm_pair.cuh"

namespace dyra {

using namespace sm100;

namespace {

__device__ __forceinline__ uint64_t kmajor_desc(uint32_t base, int ks) {
  // K-major, 128-byte swizzle: rows of 64 bf16, 8-row atoms 1024 bytes apart;
  // the k-th group of 16 elements starts 32 bytes further into each row.
  return smem_desc(base + static_cast<uint32_t>(ks) * 32u, 16u, 1024u, kLayoutSw128);
}

__device__ __forceinline__ float f32(uint32_t u) { return __uint_as_float(u); }

// Write eight fp32 accumulator values as one 16-byte bf16 vector.
__device__ __forceinline__ void store8_bf16(void* dst, const uint32_t (&v)[32], int g) {
  st_global_v4(dst, pack_bf16x2(f32(v[8 * g + 0]), f32(v[8 * g + 1])),
               pack_bf16x2(f32(v[8 * g + 2]), f32(v[8 * g + 3])),
               pack_bf16x2(f32(v[8 * g + 4]), f32(v[8 * g + 5])),
               pack_bf16x2(f32(v[8 * g + 6]), f32(v[8 * g + 7])));
}

__device__ __forceinline__ int ceil_div_dev(int a, int b) { return (a + b - 1) / b; }

// Epilogue helper: writes one 128 x 64 box of the accumulator (TMEM columns
// col0 .. col0+63 of this thread's row) as bf16 through a 128-byte-swizzled
// shared-memory box and a TMA store at (x, y) of `tmap`. Two boxes rotate: a
// box is rewritten only after the store issued two boxes earlier has read it.
// All 128 epilogue threads call it; thread 0 issues the stores. With `bias`
// (ncols entries, ncols a multiple of 8) bias[x + j] is added to column j of
// the box in fp32 before the rounding; columns at or beyond ncols read none.
constexpr uint32_t kStoreBoxBytes = 128u * 128u;  // 128 rows x 64 bf16
constexpr uint32_t kStoreBoxes = 2;

// With LO set, the box receives the low part of each value instead,
// bf16(v - bf16(v)): the two boxes together carry v to about 16 bits. BIAS
// compiles the bias add in (the callers without one keep the plain loop).
template <bool LO = false, bool BIAS = false>
__device__ __forceinline__ void store_box_bf16(uint32_t tacc, int col0, const void* tmap, int x,
                                               int y, EpiCtx& e,
                                               const __nv_bfloat16* bias = nullptr,
                                               int ncols = 0) {
  const uint32_t buf = e.counter % kStoreBoxes;
  ++e.counter;
  // the box's 64 bias values (8 columns per load, all inside or all beyond
  // ncols) are loaded first, so that their latency passes during the TMEM
  // loads and the wait for the store buffer
  uint4 bq[BIAS ? 8 : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = x + j * 8;
      bq[j] = c < ncols ? __ldg(reinterpret_cast<const uint4*>(bias + c)) : make_uint4(0, 0, 0, 0);
    }
  }
  // both TMEM loads in flight before one wait, and during the wait for the
  // store buffer
  uint32_t vv[2][32];
  tmem_ld_32x32b_x32(tacc + col0, vv[0]);
  tmem_ld_32x32b_x32(tacc + col0 + 32, vv[1]);
  if (e.tid == 0) tma_store_wait_read<kStoreBoxes - 1>();
  named_bar_sync(1, 128);
  uint8_t* sbuf = e.smem + buf * kStoreBoxBytes;
  tmem_ld_wait();
  if constexpr (BIAS) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        const uint4& b8 = bq[half * 4 + ch];
        const uint32_t w[4] = {b8.x, b8.y, b8.z, b8.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t& v0 = vv[half][8 * ch + 2 * j];
          uint32_t& v1 = vv[half][8 * ch + 2 * j + 1];
          v0 = __float_as_uint(f32(v0) + __uint_as_float(w[j] << 16));
          v1 = __float_as_uint(f32(v1) + __uint_as_float(w[j] & 0xffff0000u));
        }
      }
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      const int chunk = half * 4 + ch;
      const uint32_t off =
          static_cast<uint32_t>(e.row) * 128u + static_cast<uint32_t>((chunk ^ (e.row & 7)) * 16);
      auto val = [&](int c) {
        const float v = f32(vv[half][8 * ch + c]);
        return LO ? v - __bfloat162float(__float2bfloat16_rn(v)) : v;
      };
      uint4 q;
      q.x = pack_bf16x2(val(0), val(1));
      q.y = pack_bf16x2(val(2), val(3));
      q.z = pack_bf16x2(val(4), val(5));
      q.w = pack_bf16x2(val(6), val(7));
      *reinterpret_cast<uint4*>(sbuf + off) = q;
    }
  }
  fence_async_shared();
  named_bar_sync(1, 128);
  if (e.tid == 0) {
    tma_store_2d(tmap, e.smem_u32 + buf * kStoreBoxBytes, x, y);
    tma_store_commit();
  }
}


__device__ __forceinline__ void store_drain(EpiCtx& e) {
  if (e.tid == 0) tma_store_wait_all();
}

// ------------------------------------------------------------- host side ----

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

uint32_t pow2_at_least(uint32_t x) {
  uint32_t v = 32;
  while (v < x) v <<= 1;
  return v;
}

// Fill the shared part of the launch parameters; returns dynamic smem bytes
// or 0 if the tile shape does not fit.
template <class Pol>
uint32_t setup_common(GemmCommon& c, int num_tiles, uint32_t a_bytes, uint32_t b_bytes,
                      int mma_n, bool a_mn, bool b_mn, int* status, const DeviceInfo& dev,
                      int smem_cap = 0) {
  c.num_tiles = num_tiles;
  c.defer_wait = 0;
  c.trigger_after_wait = 0;
  c.b_parts = 1;
  c.b_part_desc = 0;
  c.wait_ns = sm100::kWaitLimitNs;
  c.early = 0;
  c.a_stage_bytes = a_bytes;
  c.b_stage_bytes = b_bytes;
  c.acc_cols = static_cast<uint32_t>((mma_n + 31) / 32 * 32);
  c.tmem_cols = pow2_at_least(2 * c.acc_cols);
  if (c.tmem_cols > 512) return 0;
  c.idesc = idesc_bf16(128, mma_n, a_mn, b_mn);
  c.status = status;
  c.trace = nullptr;
  const uint32_t fixed = gemm_smem_bytes(0, a_bytes, b_bytes, Pol::kEpiSmemBytes);
  const int full = (dev.max_smem_optin - static_cast<int>(fixed)) / static_cast<int>(a_bytes + b_bytes);
  int stages = full;
  if (smem_cap > 0) {
    // a cap that would leave fewer than 3 stages is not worth its room
    const int capped = (std::min(smem_cap, dev.max_smem_optin) - static_cast<int>(fixed)) /
                       static_cast<int>(a_bytes + b_bytes);
    if (capped >= 3) stages = capped;
  }
  stages = std::min(stages, kMaxStages);
  if (stages < 2) return 0;
  c.stages = stages;
  return gemm_smem_bytes(stages, a_bytes, b_bytes, Pol::kEpiSmemBytes);
}

template <class Pol>
int launch_gemm(const typename Pol::Params& p, uint32_t smem, const DeviceInfo& dev,
                cudaStream_t s, bool pdl, int cluster = 1) {
  if (p.c.num_tiles <= 0) return 0;
  auto kfn = umma_gemm_kernel<Pol>;
  static KernelSetup setup;
  if (raise_smem(kfn, setup, dev.device, smem)) return -1;
  cudaLaunchConfig_t cfg = {};
  // with clusters every CTA takes exactly one tile (the grid is the tile count)
  cfg.gridDim = dim3(static_cast<unsigned>(
      cluster > 1 ? p.c.num_tiles : std::min(p.c.num_tiles, dev.sm_count)));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  if (cluster > 1) {
    if (p.c.num_tiles % cluster != 0) return -1;
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(na);
  return cudaLaunchKernelEx(&cfg, kfn, p) == cudaSuccess ? 0 : -1;
}

template <class Pol>
int launch_gemm_pair(const typename Pol::Params& p, uint32_t smem, const DeviceInfo& dev,
                     cudaStream_t s, bool pdl) {
  if (p.c.num_tiles <= 0) return 0;
  auto kfn = umma_gemm_pair_kernel<Pol>;
  static KernelSetup setup;  // occupancy: resident pairs at the configured size
  const int d = dev.device;
  if (raise_smem(kfn, setup, d, smem)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(64 + 32 * EpiWarps<Pol>::value);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  if (setup.occupancy[d].load() < 1) {  // (a CTA per SM at any of the sizes)
    cfg.gridDim = dim3(2 * (dev.sm_count / 2));
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kfn, &cfg) != cudaSuccess || clusters < 1) {
      cudaGetLastError();
      clusters = dev.sm_count / 2;
    }
    setup.occupancy[d].store(clusters);
  }
  const int max_pairs = setup.occupancy[d].load();
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(p.c.num_tiles, max_pairs)));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kfn, p) == cudaSuccess ? 0 : -1;
}

}  // namespace

}  // namespace dyra
