// layers_moe_umma.cu - bf16 experts for up to 64 tokens on tcgen05 tensor cores,
// in two kernels of stream_gemm.cuh's form and one that joins their parts.
//
// The layer is bound by reading the weights of the experts its tokens reach, so
// each is read once and meets all tokens of the call: the tokens are the N side
// of the MMAs (16 to 64 columns), whichever of them name the expert. A column of
// a token that does not name it is computed and left unused; it touches no other
// column, so neither its values nor a foreign expert's can leak into a result.
//   gate-up  hidden[a][n][f] = act(Wg_e x_n) * (Wu_e x_n) for the a-th reached
//            expert e: tiles of 64 gate rows over the 64 up rows of the same f
//   down     y[n][d] = sum over a of w(n, e) (Wd_e hidden[a][n])[d]: tiles of 128
//            rows d whose steps run through the reached experts; the weights are
//            applied in fp32 at the end of each expert's run, the running sum of
//            a CTA's share of a tile stays in registers
//   join     the shares' sums, in order, and the residual
// A few tiles hold all of down's steps, so each has many parts (10 of 64 columns
// at 64 tokens over 128 experts of 2048 x 1024): summed by the last CTA to arrive
// they took about 20 us, spread over a grid of their own 3.
// The down kernel starts while the gate-up kernel drains: its weights do not
// depend on it and are copied before the wait.
#include <algorithm>

#include "layers.h"
#include "layers_math.cuh"
#include "stream_gemm.cuh"

namespace dyra {

namespace {

struct MoeTables {
  const int* ids;        // N x top_k
  const float* weights;  // N x top_k
  int N, top_k, experts;
};

// Block-wide: the experts that the ids name, in order of their index. list holds
// min(experts, N * top_k) entries.
struct MoeList {
  uint32_t bits[DYRA_MOE_MAX_EXPERTS / 32];
  int count;
  int pad[3];
  uint16_t list[DYRA_MOE_MAX_EXPERTS];
};

__device__ __forceinline__ void build_list(MoeList& l, const MoeTables& t) {
  constexpr int kWords = DYRA_MOE_MAX_EXPERTS / 32;
  if (threadIdx.x < kWords) l.bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < t.N * t.top_k; i += kStreamThreads) {
    const int e = t.ids[i];
    if (e >= 0 && e < t.experts) atomicOr(&l.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // one lane per word: its experts follow the words before it
    uint32_t b = threadIdx.x < kWords ? l.bits[threadIdx.x] : 0;
    int at = __popc(b);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (threadIdx.x >= o) at += v;
    }
    if (threadIdx.x == 31) l.count = at;
    at -= __popc(b);
    while (b) {
      l.list[at++] = static_cast<uint16_t>(threadIdx.x * 32 + __ffs(b) - 1);
      b &= b - 1;
    }
  }
  // the caller's block barrier publishes the list
}

// ---------------------------------------------------------------- gate-up ----
struct GateUpParams {
  StreamCommon c;
  CUtensorMap tmW;  // (d, 2 f, experts), box (64, 64, 1)
  CUtensorMap tmX;  // (d, N, 1), box (64, nb, 1)
  MoeTables t;
  int d, f, act;
  __nv_bfloat16* hidden;  // [reached expert][kMoeTokens][f]
  size_t hidden_extent;
};

struct GateUpPolicy {
  using Params = GateUpParams;
  static constexpr bool kWholeTiles = true;
  struct Acc {};
  struct Smem {
    float up[kMoeTokens][64];
    MoeList l;
  };
  static constexpr uint32_t kSmemBytes = (sizeof(Smem) + 15) / 16 * 16;
  static constexpr uint64_t kAStep = 2, kBStep = 2;
  static __device__ __forceinline__ Smem& of(uint8_t* sm) { return *reinterpret_cast<Smem*>(sm); }

  static __device__ __forceinline__ void prefetch(const Params& p) {
    tma_prefetch_desc(&p.tmW);
    tma_prefetch_desc(&p.tmX);
  }
  static __device__ __forceinline__ void setup(const Params& p, uint8_t* sm) {
    build_list(of(sm).l, p.t);
  }
  static __device__ __forceinline__ int f_tiles(const Params& p) { return ceil_div_dev(p.f, 64); }
  static __device__ __forceinline__ void shape(const Params& p, uint8_t* sm, int& tiles, int& nsub,
                                               int& ks) {
    tiles = of(sm).l.count * f_tiles(p);
    nsub = 1;
    ks = ceil_div_dev(p.d, 64);
  }
  static __device__ __forceinline__ void load_a(const Params& p, uint8_t* sm, int tile, int, int k,
                                                uint32_t dst, uint32_t bar) {
    const int a = tile / f_tiles(p), f0 = (tile - a * f_tiles(p)) * 64;
    const int e = of(sm).l.list[a];
    // a ragged last gate box reads up rows too; their products are left unused
    tma_load_3d(dst, &p.tmW, bar, k * 64, f0, e);
    tma_load_3d(dst + 8192u, &p.tmW, bar, k * 64, p.f + f0, e);
  }
  static __device__ __forceinline__ void load_b(const Params& p, uint8_t*, int, int, int k,
                                                uint32_t dst, uint32_t bar) {
    tma_load_3d(dst, &p.tmX, bar, k * 64, 0, 0);
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t a) { return kmajor_desc(a, 0); }
  static __device__ __forceinline__ uint64_t bdesc(uint32_t b) { return kmajor_desc(b, 0); }

  // The up rows (tile rows 64..127) hand their columns to the gate rows.
  static __device__ __forceinline__ void finish(const Params& p, uint8_t* sm, int tile, int row,
                                                int col, const float (&v)[32]) {
    const int a = tile / f_tiles(p), f = (tile - a * f_tiles(p)) * 64 + (row & 63);
    if (row >= 64) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < p.t.N) of(sm).up[col + i][row - 64] = v[i];
    }
    named_bar_sync(1, 128);
    if (row < 64 && f < p.f)
      with_act(p.act, [&](auto tag) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (col + i >= p.t.N) break;
          const size_t at = (static_cast<size_t>(a) * kMoeTokens + col + i) * p.f + f;
          if (!in_bounds(p.c.status, at, 1, p.hidden_extent)) continue;
          // rounded to bf16: an operand of the down product's tensor cores
          p.hidden[at] = __float2bfloat16_rn(act_f<decltype(tag)::value, true>(v[i]) *
                                             of(sm).up[col + i][row]);
        }
      });
  }
  template <class Release>
  static __device__ __forceinline__ void segment(const Params& p, uint8_t* sm, const StreamSeg& s,
                                                 int per_tile, uint32_t tacc, StreamEpi& e, Acc&,
                                                 const Release& release) {
    float* part = stream_part(p.c, static_cast<int>(blockIdx.x), s.first) + e.row;
    for (int col = 0; col < p.t.N; col += 32) {
      __syncwarp();
      uint32_t raw[32];
      tmem_ld_32x32b_x32(tacc + col, raw);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = f32(raw[i]);
      if (s.whole) {
        finish(p, sm, s.tile, e.row, col, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i < p.t.N) part[(col + i) * 128] = v[i];
      }
    }
    release();
    if (s.whole) return;
    int c0, c1;
    if (!stream_arrive(p.c, s, per_tile, e, c0, c1)) return;
    for (int col = 0; col < p.t.N; col += 32) {
      float v[32];
      stream_sum(p.c, c0, c1, e.row, col, p.t.N - col, v);
      finish(p, sm, s.tile, e.row, col, v);
    }
  }
  static __device__ __forceinline__ void nothing(const Params&, const StreamEpi&) {}
};

// ------------------------------------------------------------------- down ----
struct DownParams {
  StreamCommon c;
  CUtensorMap tmW;  // (f, d, experts), box (64, 128, 1)
  CUtensorMap tmH;  // (f, N, reached experts), box (64, nb, 1), rows kMoeTokens apart
  MoeTables t;
  int d, f;
  int* meta;  // for the join: steps, CTAs, steps of a tile
};

// The part of a tile that a CTA leaves: along the sequence of shares either the
// tile or the CTA or both go up by one from part to part, so their sum names it.
__device__ __forceinline__ float* down_part(const StreamCommon& c, int cta, int tile) {
  return c.ws + static_cast<size_t>(cta + tile) * static_cast<size_t>(c.nb) * 128;
}

struct DownPolicy {
  using Params = DownParams;
  static constexpr bool kWholeTiles = false;
  struct Acc {  // the running sums of this thread's row, column by column
    float v[kMoeTokens];
    bool fresh = true;
  };
  struct Smem {
    float w[kMoeTokens];  // of the run's expert
    int named[kMoeTokens];
    float weights[kMoeTokens * DYRA_MOE_MAX_TOP_K];
    int ids[kMoeTokens * DYRA_MOE_MAX_TOP_K];
    MoeList l;
  };
  static constexpr uint32_t kSmemBytes = (sizeof(Smem) + 15) / 16 * 16;
  static constexpr uint64_t kAStep = 2, kBStep = 2;
  static __device__ __forceinline__ Smem& of(uint8_t* sm) { return *reinterpret_cast<Smem*>(sm); }

  static __device__ __forceinline__ void prefetch(const Params& p) {
    tma_prefetch_desc(&p.tmW);
    tma_prefetch_desc(&p.tmH);
  }
  static __device__ __forceinline__ void setup(const Params& p, uint8_t* sm) {
    Smem& s = of(sm);
    for (int i = threadIdx.x; i < p.t.N * p.t.top_k; i += kStreamThreads) {
      s.ids[i] = p.t.ids[i];
      s.weights[i] = p.t.weights[i];
    }
    build_list(s.l, p.t);
  }
  static __device__ __forceinline__ void shape(const Params& p, uint8_t* sm, int& tiles, int& nsub,
                                               int& ks) {
    nsub = of(sm).l.count;
    tiles = nsub ? ceil_div_dev(p.d, 128) : 0;
    ks = ceil_div_dev(p.f, 64);
  }
  static __device__ __forceinline__ void load_a(const Params& p, uint8_t* sm, int tile, int sub,
                                                int k, uint32_t dst, uint32_t bar) {
    tma_load_3d(dst, &p.tmW, bar, k * 64, tile * 128, of(sm).l.list[sub]);
  }
  static __device__ __forceinline__ void load_b(const Params& p, uint8_t*, int, int sub, int k,
                                                uint32_t dst, uint32_t bar) {
    tma_load_3d(dst, &p.tmH, bar, k * 64, 0, sub);
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t a) { return kmajor_desc(a, 0); }
  static __device__ __forceinline__ uint64_t bdesc(uint32_t b) { return kmajor_desc(b, 0); }

  template <class Release>
  static __device__ __forceinline__ void segment(const Params& p, uint8_t* sm, const StreamSeg& s,
                                                 int per_tile, uint32_t tacc, StreamEpi& e,
                                                 Acc& acc, const Release& release) {
    Smem& t = of(sm);
    if (e.tid < p.t.N) {  // a token that names the expert twice gets both weights
      const int ex = t.l.list[s.sub];
      float w = 0.f;
      int named = 0;
      for (int k = 0; k < p.t.top_k; ++k)
        if (t.ids[e.tid * p.t.top_k + k] == ex) {
          w += t.weights[e.tid * p.t.top_k + k];
          named = 1;
        }
      t.w[e.tid] = w;
      t.named[e.tid] = named;
    }
    if (acc.fresh) {
#pragma unroll
      for (int i = 0; i < kMoeTokens; ++i) acc.v[i] = 0.f;
    }
    acc.fresh = s.last;
    named_bar_sync(1, 128);
#pragma unroll
    for (int half = 0; half < kMoeTokens / 32; ++half) {
      if (half * 32 >= p.t.N) break;
      __syncwarp();
      uint32_t raw[32];
      tmem_ld_32x32b_x32(tacc + half * 32, raw);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int col = half * 32 + i;
        // skipped, not multiplied by zero: the column may hold anything
        if (col < p.t.N && t.named[col])
          acc.v[col] = fmaf(t.w[col], f32(raw[i]), acc.v[col]);
      }
    }
    release();
    if (blockIdx.x == 0 && e.tid == 0) {
      p.meta[0] = e.total;
      p.meta[1] = e.grid;
      p.meta[2] = per_tile;
    }
    if (!s.last) return;
    float* part = down_part(p.c, static_cast<int>(blockIdx.x), s.tile) + e.row;
#pragma unroll
    for (int i = 0; i < kMoeTokens; ++i)
      if (i < p.t.N) part[i * 128] = acc.v[i];
  }
  // no token names an expert
  static __device__ __forceinline__ void nothing(const Params& p, const StreamEpi& e) {
    if (blockIdx.x == 0 && e.tid == 0) p.meta[0] = 0;
  }
};

// ------------------------------------------------------------------- join ----
// Y[n][8 o ..] = the sum, in the CTAs' order, of the down tile's parts of that
// column, plus the residual: eight rows of a token per thread.
__global__ void __launch_bounds__(128)
    moe_join_kernel(const __grid_constant__ StreamCommon c, const int* meta,
                    const __nv_bfloat16* residual, __nv_bfloat16* Y, int N, int d) {
  pdl_wait();
  pdl_launch_dependents();
  const int octets = d / 8;
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i >= octets * N) return;
  const int n = i / octets, o = i - n * octets;
  const size_t at = static_cast<size_t>(n) * d + static_cast<size_t>(o) * 8;
  if (!in_bounds(c.status, at, 8, static_cast<size_t>(N) * d)) return;
  uint4 r = make_uint4(0, 0, 0, 0);
  if (residual) r = *reinterpret_cast<const uint4*>(residual + at);
  const int total = meta[0];
  float v[8] = {};
  if (total > 0) {
    const int grid = meta[1], per_tile = meta[2], tile = o / 16;
    const int c0 = stream_owner(tile * per_tile, total, grid);
    const int c1 = stream_owner(tile * per_tile + per_tile - 1, total, grid);
    const size_t off = static_cast<size_t>(n) * 128 + (o % 16) * 8;
    constexpr int kFlight = 6;  // parts in flight
    for (int q0 = c0; q0 <= c1; q0 += kFlight) {
      float4 x[kFlight][2];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int q = min(q0 + u, c1);
        const float4* part = reinterpret_cast<const float4*>(down_part(c, q, tile) + off);
        x[u][0] = __ldcg(part);
        x[u][1] = __ldcg(part + 1);
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        if (q0 + u <= c1) {
          v[0] += x[u][0].x, v[1] += x[u][0].y, v[2] += x[u][0].z, v[3] += x[u][0].w;
          v[4] += x[u][1].x, v[5] += x[u][1].y, v[6] += x[u][1].z, v[7] += x[u][1].w;
        }
    }
  }
  if (residual) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] += __uint_as_float(w[j] << 16);
      v[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  *reinterpret_cast<uint4*>(Y + at) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7]));
}

bool encode_3d(CUtensorMap* tm, const void* base, int64_t len, int64_t rows, int64_t slabs,
               int64_t slab_rows, uint32_t box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(len), static_cast<uint64_t>(rows),
                            static_cast<uint64_t>(slabs)};
  const uint64_t strides[2] = {static_cast<uint64_t>(len) * 2,
                               static_cast<uint64_t>(len) * 2 * static_cast<uint64_t>(slab_rows)};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_tmap_bf16(tm, base, 3, dims, strides, box, 128);
}

}  // namespace

int moe_reached_max(const MoeShape& m) { return std::min(m.experts, kMoeTokens * m.top_k); }

// the gate-up tiles' arrival counters, then the join's three words
int moe_counters(const MoeShape& m) { return moe_reached_max(m) * ceil_div(m.f, 64) + 4; }

// two parts per CTA of gate-up, or down's: one per CTA and tile border
size_t moe_ws_bytes(const MoeShape& m, const DeviceInfo& dev) {
  const size_t parts = static_cast<size_t>(dev.sm_count) + std::max(dev.sm_count, ceil_div(m.d, 128));
  return parts * kMoeTokens * 128 * sizeof(float);
}

int launch_moe_experts_umma(const MoeShape& m, const __nv_bfloat16* X, const int* ids,
                            const float* weights, const __nv_bfloat16* Wgu,
                            const __nv_bfloat16* Wd, const __nv_bfloat16* residual,
                            __nv_bfloat16* Y, int N, __nv_bfloat16* hidden, float* ws,
                            int* counters, int* status, unsigned long long wait_ns,
                            const DeviceInfo& dev, cudaStream_t s) {
  const int nb = ceil_div(N, 16) * 16;
  const int reached = std::min(m.experts, N * m.top_k);
  const MoeTables t{ids, weights, N, m.top_k, m.experts};
  GateUpParams g;
  g.t = t;
  g.d = m.d;
  g.f = m.f;
  g.act = m.act;
  g.hidden = hidden;
  g.hidden_extent = static_cast<size_t>(moe_reached_max(m)) * kMoeTokens * m.f;
  DownParams w;
  w.t = t;
  w.d = m.d;
  w.f = m.f;
  w.meta = counters + moe_reached_max(m) * ceil_div(m.f, 64);
  if (!encode_3d(&g.tmW, Wgu, m.d, 2 * static_cast<int64_t>(m.f), m.experts,
                 2 * static_cast<int64_t>(m.f), 64) ||
      !encode_3d(&g.tmX, X, m.d, N, 1, N, static_cast<uint32_t>(nb)) ||
      !encode_3d(&w.tmW, Wd, m.f, m.d, m.experts, m.d, 128) ||
      !encode_3d(&w.tmH, hidden, m.f, N, reached, kMoeTokens, static_cast<uint32_t>(nb)))
    return -2;
  const uint32_t smem_g =
      stream_setup<GateUpPolicy>(g.c, nb, false, false, ws, counters, status, wait_ns, dev);
  const uint32_t smem_d =
      stream_setup<DownPolicy>(w.c, nb, false, false, ws, nullptr, status, wait_ns, dev);
  if (!smem_g || !smem_d) return -3;
  w.c.late_b = 1;
  if (stream_launch<GateUpPolicy>(g, smem_g, dev, s)) return -1;
  if (stream_launch<DownPolicy>(w, smem_d, dev, s)) return -1;
  const dim3 grid(static_cast<unsigned>(ceil_div(static_cast<int64_t>(m.d) / 8 * N, 128)));
  return launch_dependent(moe_join_kernel, grid, dim3(128), 0, 1, s, w.c,
                          static_cast<const int*>(w.meta), residual, Y, N, m.d);
}

}  // namespace dyra
