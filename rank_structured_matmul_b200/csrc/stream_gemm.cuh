// stream_gemm.cuh - tensor-core products that are bound by reading one operand
// once: a few columns (tokens) against long rows of weights.
//
// D tile = 128 rows of A (weights) x nb columns of B (tokens), accumulated over
// steps of 64 k. All tiles' steps form one sequence, and the grid's CTAs take
// equal contiguous shares of it (within one step), whatever the tile count: the 32
// down tiles of one token on two experts of 4096 x 14336 keep all 148 SMs reading to
// the end, where a tile per CTA would leave most of them idle. A tile that
// a share's border cuts is summed from the fp32 parts its CTAs leave in a
// workspace, in the order of the CTAs, by the one that arrives last (or, where a
// tile has many parts, by a grid that follows): no CTA waits for another, and the
// result does not depend on who is last.
//
// Roles as in umma_gemm.cuh: warp 0 copies (TMA, a ring of up to 12 stages),
// warp 1 issues the MMAs into one of two accumulators, warps 2..5 take the
// accumulators. Waits are bounded in the same way.
//
// A tile's steps may fall into `nsub` equal runs (an expert each); the
// accumulator goes to the epilogue at the end of every run. A policy supplies
//   struct Params { StreamCommon c; ... };
//   static constexpr uint32_t kSmemBytes;   // its own shared memory, a multiple of 16
//   static constexpr bool kWholeTiles;      // tiles are left whole where that is cheaper
//   struct Acc;                             // an epilogue thread's state between segments
//   static void prefetch(p);
//   static void setup(p, sm);               // all threads, before the roles start
//   static void shape(p, sm, int& tiles, int& nsub, int& ks);
//   static void load_a / load_b(p, sm, tile, sub, k, dst, bar);
//   static uint64_t adesc / bdesc(address);   // of the first of a step's four MMAs
//   static constexpr uint64_t kAStep, kBStep;  // from one MMA's descriptor to the next
//   static void segment(p, sm, seg, per_tile, tacc, epi, Acc&, release);
//   static void nothing(p, epi);            // there are no steps at all
#pragma once

#include "layers.h"
#include "umma_common.cuh"

namespace dyra {

constexpr int kStreamThreads = 192;
constexpr int kStreamMaxStages = 12;
constexpr int kStreamMaxNb = 128;
constexpr uint32_t kStreamABytes = 128u * 128u;  // 128 rows x 64 bf16

constexpr int kJoinSteps = 8;

struct StreamCommon {
  int nb;              // columns of a tile: a multiple of 16, at most 128
  int stages;
  uint32_t b_bytes;    // nb x 64 bf16
  uint32_t acc_cols, tmem_cols, idesc;
  int min_steps;       // a CTA's share is at least this many steps
  int* status;
  float* ws;           // parts: [CTA][2][nb][128]
  int* counters;       // arrivals per tile, zero between launches
  // 1: launched behind a grid that writes B, with everything else complete at
  // launch: A is copied before the dependency wait, B after it
  int late_b;
  unsigned long long wait_ns;  // limit of one pipeline wait; drains keep kWaitLimitNs
};

// A run of steps [k0, k0 + n) of run `sub` of `tile`.
struct StreamSeg {
  int tile, sub, k0, n;
  bool first;  // the tile's first step is in this CTA's share
  bool whole;  // (at the tile's last segment here) all its steps are
  bool last;   // no further segment of this tile follows in this CTA
};

struct StreamWalk {
  int i, i1, per_tile, ks, tile_start;
  __device__ __forceinline__ bool next(StreamSeg& s) {
    if (i >= i1) return false;
    s.tile = i / per_tile;
    const int r = i - s.tile * per_tile;
    s.sub = r / ks;
    s.k0 = r - s.sub * ks;
    s.n = min(ks - s.k0, i1 - i);
    const int t0 = s.tile * per_tile, t1 = t0 + per_tile;
    s.first = t0 >= tile_start;
    i += s.n;
    s.last = i >= i1 || i == t1;
    s.whole = s.first && i == t1;
    return true;
  }
};

struct StreamEpi {
  int row;   // tile row of this thread, 0..127
  int tid;   // 0..127
  int total, grid;  // steps and CTAs taking part
  volatile int* flag;  // shared word of the last-arrival vote
};

__host__ __device__ inline uint32_t stream_smem_bytes(int stages, uint32_t b_bytes,
                                                      uint32_t pol_bytes) {
  return 1024u + static_cast<uint32_t>(stages) * (kStreamABytes + b_bytes) + pol_bytes + 512u;
}

// CTA whose share holds step i.
__device__ __forceinline__ int stream_owner(int i, int total, int grid) {
  // largest c with c * total / grid <= i
  return static_cast<int>(((static_cast<long long>(i) + 1) * grid + total - 1) / total) - 1;
}

__device__ __forceinline__ float* stream_part(const StreamCommon& c, int cta, bool first) {
  return c.ws + (static_cast<size_t>(cta) * 2 + (first ? 1 : 0)) * static_cast<size_t>(c.nb) * 128;
}

// This CTA's part of the tile is in the workspace: true for the last CTA of the
// tile to arrive, which then sums the parts of CTAs c0 .. c1.
__device__ __forceinline__ bool stream_arrive(const StreamCommon& c, const StreamSeg& s,
                                              int per_tile, const StreamEpi& e, int& c0, int& c1) {
  c0 = stream_owner(s.tile * per_tile, e.total, e.grid);
  c1 = stream_owner(s.tile * per_tile + per_tile - 1, e.total, e.grid);
  __threadfence();
  named_bar_sync(1, 128);
  if (e.tid == 0) {
    const int old = atomicAdd(c.counters + s.tile, 1);
    const bool last = old == c1 - c0;
    if (last) c.counters[s.tile] = 0;
    *e.flag = last;
  }
  named_bar_sync(1, 128);
  const bool last = *e.flag != 0;
  named_bar_sync(1, 128);  // the word may be written again
  if (last) __threadfence();
  return last;
}

// v[i] = sum over the parts, in order, of column col0 + i (i < n) of this row.
template <int NV>
__device__ __forceinline__ void stream_sum(const StreamCommon& c, int c0, int c1, int row,
                                           int col0, int n, float (&v)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.f;
  for (int cta = c0; cta <= c1; ++cta) {
    const float* part = stream_part(c, cta, cta == c0) + static_cast<size_t>(col0) * 128 + row;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i < n) v[i] += __ldcg(part + i * 128);
  }
}

template <class Pol>
__global__ void __launch_bounds__(kStreamThreads, 1)
    stream_kernel(const __grid_constant__ typename Pol::Params p) {
  extern __shared__ uint8_t smem_raw[];
  const StreamCommon& c = p.c;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  const int S = c.stages;
  const uint32_t sA = sbase, sB = sA + static_cast<uint32_t>(S) * kStreamABytes;
  const uint32_t off_pol = static_cast<uint32_t>(S) * (kStreamABytes + c.b_bytes);
  uint8_t* const sm = smem + off_pol;
  const uint32_t sBar = sbase + off_pol + Pol::kSmemBytes;
  auto full_bar = [&](int s) { return sBar + 8u * s; };
  auto empty_bar = [&](int s) { return sBar + 8u * (kStreamMaxStages + s); };
  auto tfull_bar = [&](int i) { return sBar + 8u * (2 * kStreamMaxStages + i); };
  auto tempty_bar = [&](int i) { return sBar + 8u * (2 * kStreamMaxStages + 2 + i); };
  const uint32_t fin_bar = sBar + 8u * (2 * kStreamMaxStages + 4);
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + off_pol + Pol::kSmemBytes +
                                                8 * (2 * kStreamMaxStages + 5));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(words + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 4);
    }
    mbar_init(fin_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) Pol::prefetch(p);
  if (warp == 1) {
    tmem_alloc(smem_u32(words), c.tmem_cols);
    tmem_relinquish();
  }
  // late_b: the grid before this one let it start only after its own wait, so
  // whatever the grids before that one wrote is visible already
  if (!c.late_b) pdl_wait();
  Pol::setup(p, sm);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // must stay behind the wait above: a late_b grid reads before its own
  if (!c.late_b) pdl_launch_dependents();
  const uint32_t tmem = words[0];

  int tiles, nsub, ks;
  Pol::shape(p, sm, tiles, nsub, ks);
  const int per_tile = nsub * ks;
  const int total = tiles * per_tile;
  const int all = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  // whole tiles where the fullest CTA then has at most kJoinSteps more steps than
  // its share: joining the parts of a tile takes about as long as those
  const bool cut = !Pol::kWholeTiles ||
                   (tiles + all - 1) / all * per_tile > (total + all - 1) / all + kJoinSteps;
  const int grid = cut ? max(1, min(all, total / c.min_steps)) : min(all, max(1, tiles));
  const int units = cut ? total : tiles, unit = cut ? 1 : per_tile;
  StreamWalk walk;
  walk.per_tile = per_tile;
  walk.ks = ks;
  const bool works = cta < grid && total > 0;
  walk.i = walk.tile_start =
      works ? static_cast<int>(static_cast<long long>(cta) * units / grid) * unit : 0;
  walk.i1 = works ? static_cast<int>(static_cast<long long>(cta + 1) * units / grid) * unit : 0;

  WaitCtx w{abort_flag, c.status, c.wait_ns};
  uint32_t last_phase[kStreamMaxStages];
  uint32_t issued = 0;
  StreamSeg seg;

  if (warp == 0) {
    if (elect_one_sync()) {
      int pre = 0;  // stages whose A copy was issued before the dependency wait
      if (c.late_b) {
        StreamWalk early = walk;
        while (pre < S && early.next(seg))
          for (int j = 0; j < seg.n && pre < S; ++j, ++pre) {
            mbar_arrive_expect_tx(full_bar(pre), kStreamABytes + c.b_bytes);
            Pol::load_a(p, sm, seg.tile, seg.sub, seg.k0 + j, sA + pre * kStreamABytes,
                        full_bar(pre));
          }
        pdl_wait();
        pdl_launch_dependents();
      }
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && walk.next(seg)) {
        for (int j = 0; j < seg.n; ++j, ++count) {
          const int k = seg.k0 + j;
          if (count >= pre) {
            if (!mbar_wait(empty_bar(stage), phase ^ 1u, w)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(full_bar(stage), kStreamABytes + c.b_bytes);
            Pol::load_a(p, sm, seg.tile, seg.sub, k, sA + stage * kStreamABytes, full_bar(stage));
          }
          Pol::load_b(p, sm, seg.tile, seg.sub, k, sB + stage * c.b_bytes, full_bar(stage));
          issued |= 1u << stage;
          last_phase[stage] = phase;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one_sync()) {
      int stage = 0, local = 0;
      uint32_t phase = 0;
      while (walk.next(seg)) {
        const int acc = local & 1;
        if (!mbar_wait(tempty_bar(acc), ((local >> 1) & 1) ^ 1u, w)) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc) * c.acc_cols;
        bool ok = true;
        for (int j = 0; j < seg.n; ++j) {
          const uint64_t a0 = Pol::adesc(sA + stage * kStreamABytes);
          const uint64_t b0 = Pol::bdesc(sB + stage * c.b_bytes);
          if (!mbar_wait(full_bar(stage), phase, w)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // the zero fill beyond K makes a short last step's MMAs add nothing
          issue_stage<false>(d, a0, Pol::kAStep, b0, Pol::kBStep, c.idesc, 4, j == 0);
          mma_commit(empty_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(tfull_bar(acc));
        ++local;
      }
      mma_commit(fin_bar);
      (void)mbar_wait_until(fin_bar, 0, globaltimer_ns() + kWaitLimitNs);
    }
  } else {
    // residuals and the workspace may be touched by the grid before this one
    if (c.late_b) pdl_wait();
    StreamEpi e;
    const int quad = warp & 3;
    e.row = quad * 32 + lane;
    e.tid = threadIdx.x - 64;
    e.total = total;
    e.grid = grid;
    e.flag = reinterpret_cast<volatile int*>(words + 2);
    typename Pol::Acc acc_state;
    int local = 0;
    while (walk.next(seg)) {
      const int acc = local & 1;
      // all four warps go on or none: they meet at barriers in segment(), and
      // what the segment before left in shared memory has been read here
      if (!all_threads(1, 128, mbar_wait(tfull_bar(acc), (local >> 1) & 1, w))) break;
      tc_fence_after();
      const uint32_t tacc = tmem + static_cast<uint32_t>(acc) * c.acc_cols +
                            (static_cast<uint32_t>(quad * 32) << 16);
      auto release = [&] {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
      };
      Pol::segment(p, sm, seg, per_tile, tacc, e, acc_state, release);
      ++local;
    }
    if (total == 0) Pol::nothing(p, e);
  }
  __syncwarp();
  block_sync_all();
  if (warp == 0 && issued && *abort_flag) {
    const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
    for (int s = 0; s < S; ++s)
      if (issued & (1u << s)) (void)mbar_wait_until(full_bar(s), last_phase[s], deadline);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, c.tmem_cols);
  }
}

// The same product with each tile on a cluster of its own: the cluster's CTAs
// take equal shares of the tile's steps, leave their fp32 parts in their shared
// memory (the operand stages, free by then) and each sums and finishes a share of
// the columns over all parts, in CTA order, through distributed shared memory.
// Where a tile needs several CTAs and has many columns this is the cheaper way to
// join them: the parts of 64 columns from 16 CTAs took one CTA of the kernel
// above 45 us to sum. One tile per cluster, at most as many CTAs as steps. Of a
// policy it takes prefetch, adesc, bdesc, kAStep and kBStep as above, and
//   static int steps(p);
//   static void load_a / load_b(p, tile, k, dst, bar);
//   static int columns(p, tile);  // of the tile that exist
//   static void finish8(p, tile, octet, col, float (&v)[8]);  // rows 8 octet ..
template <class Pol>
__global__ void __launch_bounds__(kStreamThreads, 1)
    split_kernel(const __grid_constant__ typename Pol::Params p, int cs) {
  extern __shared__ uint8_t smem_raw[];
  const StreamCommon& c = p.c;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  const int S = c.stages;
  const uint32_t sA = sbase, sB = sA + static_cast<uint32_t>(S) * kStreamABytes;
  const uint32_t off_bar = static_cast<uint32_t>(S) * (kStreamABytes + c.b_bytes);
  const uint32_t sBar = sbase + off_bar;
  auto full_bar = [&](int s) { return sBar + 8u * s; };
  auto empty_bar = [&](int s) { return sBar + 8u * (kStreamMaxStages + s); };
  const uint32_t done_bar = sBar + 8u * (2 * kStreamMaxStages);
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + off_bar + 8 * (2 * kStreamMaxStages + 1));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(words + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / cs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) Pol::prefetch(p);
  if (warp == 1) {
    tmem_alloc(smem_u32(words), c.tmem_cols);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = words[0];
  const int ks = Pol::steps(p);
  const int k0 = static_cast<int>(static_cast<long long>(rank) * ks / cs);
  const int k1 = static_cast<int>(static_cast<long long>(rank + 1) * ks / cs);
  WaitCtx w{abort_flag, c.status, c.wait_ns};
  uint32_t last_phase[kStreamMaxStages];
  uint32_t issued = 0;

  if (warp == 0) {
    if (elect_one_sync()) {
      int stage = 0;
      uint32_t phase = 0;
      for (int k = k0; k < k1; ++k) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, w)) break;
        mbar_arrive_expect_tx(full_bar(stage), kStreamABytes + c.b_bytes);
        Pol::load_a(p, tile, k, sA + stage * kStreamABytes, full_bar(stage));
        Pol::load_b(p, tile, k, sB + stage * c.b_bytes, full_bar(stage));
        issued |= 1u << stage;
        last_phase[stage] = phase;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one_sync()) {
      int stage = 0;
      uint32_t phase = 0;
      for (int k = k0; k < k1; ++k) {
        const uint64_t a0 = Pol::adesc(sA + stage * kStreamABytes);
        const uint64_t b0 = Pol::bdesc(sB + stage * c.b_bytes);
        if (!mbar_wait(full_bar(stage), phase, w)) break;
        tc_fence_after();
        issue_stage<false>(tmem, a0, Pol::kAStep, b0, Pol::kBStep, c.idesc, 4, k == k0);
        mma_commit(empty_bar(stage));
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      mma_commit(done_bar);
      (void)mbar_wait_until(done_bar, 0, globaltimer_ns() + kWaitLimitNs);
    }
  } else {
    const int quad = warp & 3, row = quad * 32 + lane;
    const bool good = all_threads(1, 128, mbar_wait(done_bar, 0, w));
    tc_fence_after();
    const int n = Pol::columns(p, tile);
    const uint32_t tacc = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* part = reinterpret_cast<float*>(smem);  // [column][128 rows]
    for (int col = 0; good && col < n; col += 32) {
      __syncwarp();
      uint32_t r[32];
      tmem_ld_32x32b_x32(tacc + col, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < n) part[(col + i) * 128 + row] = f32(r[i]);
    }
  }
  // every part is in place
  __syncwarp();
  if (cs > 1)
    cluster_sync_all();
  else
    block_sync_all();
  if (!*abort_flag) {
    // eight rows of one column at a time: 16-byte pieces of the output, a
    // column's sixteen on consecutive lanes
    const int n = Pol::columns(p, tile);
    const int c0 = rank * n / cs, c1 = (rank + 1) * n / cs;
    constexpr int kFlight = 2;  // pieces of a thread in flight
    for (int i0 = c0 * 16 + static_cast<int>(threadIdx.x); i0 < c1 * 16;
         i0 += kFlight * kStreamThreads) {
      float v[kFlight][8] = {};
      for (int q = 0; q < cs; ++q) {
        float4 x[kFlight][2];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          // beyond the share: the first piece again, unused
          const int i = i0 + u * kStreamThreads < c1 * 16 ? i0 + u * kStreamThreads : i0;
          const uint32_t at = sbase + static_cast<uint32_t>(i) * 32u;  // [column][octet][8]
          const uint32_t from = cs > 1 ? mapa_shared(at, static_cast<uint32_t>(q)) : at;
          x[u][0] = ld_shared_cluster_v4(from);
          x[u][1] = ld_shared_cluster_v4(from + 16u);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          v[u][0] += x[u][0].x, v[u][1] += x[u][0].y, v[u][2] += x[u][0].z, v[u][3] += x[u][0].w;
          v[u][4] += x[u][1].x, v[u][5] += x[u][1].y, v[u][6] += x[u][1].z, v[u][7] += x[u][1].w;
        }
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int i = i0 + u * kStreamThreads;
        if (i < c1 * 16) Pol::finish8(p, tile, i & 15, i >> 4, v[u]);
      }
    }
  }
  __syncwarp();
  if (cs > 1) cluster_sync_all();  // no CTA leaves while its part is read
  block_sync_all();
  if (warp == 0 && issued && *abort_flag) {
    const unsigned long long deadline = globaltimer_ns() + kWaitLimitNs;
    for (int s = 0; s < S; ++s)
      if (issued & (1u << s)) (void)mbar_wait_until(full_bar(s), last_phase[s], deadline);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, c.tmem_cols);
  }
}

// Fill the shared launch parameters for nb columns; the dynamic shared memory
// of a block, or 0 if it does not fit.
template <class Pol>
uint32_t stream_setup(StreamCommon& c, int nb, bool a_mn, bool b_mn, float* ws, int* counters,
                      int* status, unsigned long long wait_ns, const DeviceInfo& dev) {
  c.nb = nb;
  c.b_bytes = static_cast<uint32_t>(nb) * 128u;
  c.acc_cols = static_cast<uint32_t>((nb + 31) / 32 * 32);
  c.tmem_cols = pow2_at_least(2 * c.acc_cols);
  c.idesc = idesc_bf16(128, nb, a_mn, b_mn);
  c.min_steps = 4;
  c.status = status;
  c.ws = ws;
  c.counters = counters;
  c.late_b = 0;
  c.wait_ns = wait_ns ? wait_ns : sm100::kWaitLimitNs;
  const int fixed = static_cast<int>(stream_smem_bytes(0, c.b_bytes, Pol::kSmemBytes));
  c.stages = std::min(kStreamMaxStages, (dev.max_smem_optin - fixed) /
                                            static_cast<int>(kStreamABytes + c.b_bytes));
  if (c.stages < 2) return 0;
  return stream_smem_bytes(c.stages, c.b_bytes, Pol::kSmemBytes);
}

template <class Pol>
int stream_launch(const typename Pol::Params& p, uint32_t smem, const DeviceInfo& dev,
                  cudaStream_t s) {
  auto kfn = stream_kernel<Pol>;
  static KernelSetup setup;
  if (raise_smem(kfn, setup, dev.device, smem)) return -1;
  return launch_dependent(kfn, dim3(static_cast<unsigned>(dev.sm_count)), dim3(kStreamThreads),
                          smem, 1, s, p);
}

// split_kernel<Pol>'s record, of its launches and of the question below.
template <class Pol>
KernelSetup& split_setup() {
  static KernelSetup setup;
  return setup;
}

// Clusters of cs CTAs that can be resident at once, at a CTA per SM; 0 where that
// cannot be told.
template <class Pol>
int split_resident(int cs, const DeviceInfo& dev) {
  auto kfn = split_kernel<Pol>;
  const uint32_t smem = static_cast<uint32_t>(dev.max_smem_optin);
  int n = 0;
  if (raise_smem(kfn, split_setup<Pol>(), dev.device, smem) == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / cs * cs));
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kfn, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  return n;
}

template <class Pol>
int split_launch(const typename Pol::Params& p, int tiles, int cs, uint32_t smem,
                 const DeviceInfo& dev, cudaStream_t s) {
  auto kfn = split_kernel<Pol>;
  if (raise_smem(kfn, split_setup<Pol>(), dev.device, smem)) return -1;
  return launch_dependent(kfn, dim3(static_cast<unsigned>(tiles * cs)), dim3(kStreamThreads), smem,
                          cs, s, p, cs);
}

}  // namespace dyra
