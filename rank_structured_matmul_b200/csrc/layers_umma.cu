// layers_umma.cu - the bf16 products of the dense layer on tcgen05 tensor
// cores: fp32 accumulation in tensor memory, operands by TMA, the epilogue
// (bias, activation, residual, the kept pre-activations) on the accumulator.
#include <algorithm>
#include <atomic>

#include "layers.h"
#include "layers_math.cuh"
#include "stream_gemm.cuh"
#include "umma_common.cuh"

namespace dyra {

namespace {

// MN-major, 128-byte swizzle: 64 elements of M (or N) per 128-byte row, 8 rows
// of k per 1024-byte atom, 64-wide blocks `block` bytes apart; a k step of 16
// is 2048 bytes further.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t base, int ks) {
  return smem_desc(base + static_cast<uint32_t>(ks) * 2048u, 8192u, 1024u, kLayoutSw128);
}

// v[0..8) += the eight bf16 values of q; eight values rounded to bf16
__device__ __forceinline__ void add8(float* v, const uint4& q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] += __uint_as_float(w[j] << 16);
    v[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// ------------------------------------------------------------ CTA pairs ----
// Out tile of 256 rows (j) x bn columns (m) on a CTA pair: CTA r loads rows
// j0 + 128 r of the row operand and columns m0 + (bn / 2) r of the other, each
// K-major (one box of 64 k) or MN-major (boxes of 64 x 64 k).
struct DensePairParams {
  GemmCommon c;
  CUtensorMap tmRow;  // row operand (J x K, or K x J when MN-major)
  CUtensorMap tmCol;  // column operand (M x K, or K x M when MN-major)
  CUtensorMap tmOut;  // J x M, box (32, 128), store
  CUtensorMap tmZ;    // the same over the kept pre-activations, or the residual
  int J, M, K, bn, tiles_m;
  int act;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  // The first `whole` tiles are a pair's each; of the `tail` others each is split
  // over its steps between `split` pairs, which leave their fp32 parts in ws
  // ([tail tile][part][CTA of the pair][column / 4][128 rows] float4s); the last
  // CTA to arrive of each half tile sums them in order.
  int whole, tail, split;
  float* ws;
  int* counters;  // two per tail tile, zero between calls
};

// What a pair kernel is compiled with: the gradients' products store the
// accumulator as it is; the forward adds bias and activation, and either the
// kept pre-activations (with a residual read row by row, if there is one) or a
// residual that comes by TMA into the store boxes.
enum PairEpilogue { kPlain, kForward, kForwardZ, kForwardResidual };

// kTail: some tiles are split between pairs (Params::split > 1).
template <bool kRowMn, bool kColMn, PairEpilogue kMode, bool kTail>
struct DensePairPolicy {
  static constexpr bool kEpi = kMode != kPlain, kKeepZ = kMode == kForwardZ,
                        kTmaRes = kMode == kForwardResidual;
  using Params = DensePairParams;
  struct Tile {
    int j0, m0, k0, nk;
    int tail, part;  // tail < 0: a whole tile; nk == 0: nothing
  };
  // Four groups of four epilogue warps take the tile's 32-column store boxes in turn.
  // ViT-L fc1 (K = 1024, calls back to back on warm inputs) takes 81.0 us with one group,
  // 55.8 with two, 46.7 with four; without bias and GELU 52.1, 41.2 and 39.5 (a bf16
  // library product: 39.2), so that at this K the GELU's epilogue is still longer than
  // a tile's MMAs. A second box per group, for the residual on its way, pays for the
  // operand stage it costs: 51 -> 48 us.
  static constexpr int kEpiWarps = 16, kGroups = kEpiWarps / 4;
  static constexpr int kMaxRegs = 96;  // 576 threads
  static constexpr int kCols = 32;     // columns of a store box
  static constexpr uint32_t kBoxBytes = 128u * kCols * 2u;
  static constexpr int kBufs = kTmaRes ? 2 : 1;  // result boxes of a group
  static constexpr uint32_t kGroupBytes = (kBufs + (kKeepZ ? 1 : 0)) * kBoxBytes;
  static constexpr uint32_t kEpiSmemBytes = kGroups * kGroupBytes + 128;  // barriers, a word

  static __device__ __forceinline__ void prefetch(const Params& p) {
    tma_prefetch_desc(&p.tmRow);
    tma_prefetch_desc(&p.tmCol);
    tma_prefetch_desc(&p.tmOut);
  }
  static __device__ __forceinline__ void decode(const Params& p, int tile, Tile& t) {
    const int steps = ceil_div_dev(p.K, 64);
    t.k0 = 0;
    t.nk = steps;
    t.tail = -1;
    t.part = 0;
    if (kTail && tile >= p.whole) {
      t.tail = (tile - p.whole) / p.split;
      t.part = (tile - p.whole) - t.tail * p.split;
      t.k0 = t.part * steps / p.split;
      t.nk = (t.part + 1) * steps / p.split - t.k0;
      tile = p.whole + t.tail;
    }
    t.j0 = (tile / p.tiles_m) * 256;
    t.m0 = (tile % p.tiles_m) * p.bn;
  }
  static __device__ __forceinline__ int kiters(const Params&, const Tile& t) { return t.nk; }
  static __device__ __forceinline__ void load(const Params& p, const Tile& t, int it, uint32_t sa,
                                              uint32_t sb, uint32_t bar, uint32_t rank) {
    it += t.k0;
    const int j = t.j0 + 128 * static_cast<int>(rank);
    const int m = t.m0 + (p.bn / 2) * static_cast<int>(rank);
    if (kRowMn) {
      tma_load_2d_pair(sa, &p.tmRow, bar, j, it * 64);
      tma_load_2d_pair(sa + 8192u, &p.tmRow, bar, j + 64, it * 64);
    } else {
      tma_load_2d_pair(sa, &p.tmRow, bar, it * 64, j);
    }
    if (kColMn) {
      tma_load_2d_pair(sb, &p.tmCol, bar, m, it * 64);
      if (p.bn > 128) tma_load_2d_pair(sb + 8192u, &p.tmCol, bar, m + 64, it * 64);
    } else {
      tma_load_2d_pair(sb, &p.tmCol, bar, it * 64, m);
    }
  }
  static __device__ __forceinline__ int ksteps(const Params& p, const Tile& t, int it) {
    return min(4, ceil_div_dev(p.K - (t.k0 + it) * 64, 16));
  }
  static __device__ __forceinline__ uint64_t adesc(const Params&, uint32_t a, int ks) {
    return kRowMn ? mnmajor_desc(a, ks) : kmajor_desc(a, ks);
  }
  static __device__ __forceinline__ uint64_t bdesc(const Params&, uint32_t b, int ks) {
    return kColMn ? mnmajor_desc(b, ks) : kmajor_desc(b, ks);
  }

  // 16-byte chunk c of this thread's row in a store box (rows of 64 bytes, 64-byte
  // swizzle)
  static __device__ __forceinline__ uint4* chunk(uint8_t* box, int row, int c) {
    return reinterpret_cast<uint4*>(box + row * 64 + ((c ^ ((row >> 1) & 3)) * 16));
  }
  static __device__ __forceinline__ float4* part_of(const Params& p, const Tile& t, int part,
                                                    int rank) {
    return reinterpret_cast<float4*>(p.ws) +
           (static_cast<size_t>(t.tail * p.split + part) * 2 + rank) * (p.bn / 4) * 128;
  }
  // A tail tile's part into the workspace; true where it is the last to arrive.
  static __device__ __forceinline__ bool leave_part(const Params& p, const Tile& t, uint32_t tacc,
                                                    EpiCtx& e) {
    float4* part = part_of(p, t, t.part, e.rank);
    for (int c = e.group * 32; c < p.bn; c += 32 * kGroups) {
      __syncwarp();
      uint32_t raw[32];
      tmem_ld_32x32b_x32(tacc + c, raw);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        part[(c / 4 + q) * 128 + e.row] = make_float4(f32(raw[4 * q]), f32(raw[4 * q + 1]),
                                                      f32(raw[4 * q + 2]), f32(raw[4 * q + 3]));
    }
    volatile int* last = reinterpret_cast<volatile int*>(e.smem + kGroups * kGroupBytes + 64);
    __threadfence();
    named_bar_sync(kGroups + 1, 32 * kEpiWarps);
    if (e.group == 0 && e.tid == 0) {
      int* counter = p.counters + 2 * t.tail + e.rank;
      const int old = atomicAdd(counter, 1);
      if (old == p.split - 1) *counter = 0;
      *last = old == p.split - 1;
    }
    named_bar_sync(kGroups + 1, 32 * kEpiWarps);
    const bool is_last = *last != 0;
    named_bar_sync(kGroups + 1, 32 * kEpiWarps);  // the word may be written again
    if (is_last) __threadfence();
    return is_last;
  }
  // raw = the sum of the parts' columns col .. col + 7 of this row, in order
  static __device__ __forceinline__ void sum_parts(const Params& p, const Tile& t, int col,
                                                   const EpiCtx& e, uint32_t (&raw)[8]) {
    float v[8] = {};
    const float4* from = part_of(p, t, 0, e.rank) + (col / 4) * 128 + e.row;
    const size_t stride = static_cast<size_t>(2) * (p.bn / 4) * 128;  // from part to part
    for (int part = 0; part < p.split; part += 4) {
      float4 x[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4* at = from + min(part + u, p.split - 1) * stride;
        x[u][0] = __ldcg(at);
        x[u][1] = __ldcg(at + 128);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (part + u < p.split) {
          v[0] += x[u][0].x, v[1] += x[u][0].y, v[2] += x[u][0].z, v[3] += x[u][0].w;
          v[4] += x[u][1].x, v[5] += x[u][1].y, v[6] += x[u][1].z, v[7] += x[u][1].w;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) raw[j] = __float_as_uint(v[j]);
  }
  // Eight columns at a time, in a loop: a box in straight-line code is some 20 KB with
  // the activation and runs out of the instruction caches. The next columns are on
  // their way from tensor memory meanwhile.
  static __device__ __forceinline__ void epilogue(const Params& p, const Tile& t, uint32_t tacc,
                                                  EpiCtx& e) {
    const bool summed = kTail && t.tail >= 0;
    if (summed && !leave_part(p, t, tacc, e)) return;
    const int y0 = t.j0 + 128 * e.rank, row = y0 + e.row;
    const int nbox = (min(p.bn, p.M - t.m0) + kCols - 1) / kCols;
    uint8_t* const box = e.smem + e.group * kGroupBytes;
    const uint32_t box_u32 = e.smem_u32 + e.group * kGroupBytes;
    const int bar = 1 + e.group;
    // kKeepZ: the residual by plain loads, 16 bytes of this thread's row
    const bool has_r = kKeepZ && p.residual != nullptr && row < p.J;
    // kTmaRes: the group's boxes alternate between its two buffers; a box's
    // residual is on its way while the box before it is finished. The buffers'
    // barriers are made at the group's first box.
    const uint32_t rbar = e.smem_u32 + kGroups * kGroupBytes + e.group * 16u;
    auto load_residual = [&](int b, uint32_t n) {  // thread 0: box b as the group's n-th
      tma_store_wait_read<0>();                    // the buffer's last store has been read
      const uint32_t buf = n % kBufs;
      mbar_arrive_expect_tx(rbar + 8u * buf, kBoxBytes);
      tma_load_2d(box_u32 + buf * kBoxBytes, &p.tmZ, rbar + 8u * buf, t.m0 + b * kCols, y0);
    };
    if (kTmaRes && e.tid == 0 && e.group < nbox) {
      if (e.counter == 0) {
        mbar_init(rbar, 1);
        mbar_init(rbar + 8u, 1);
        fence_barrier_init();
      }
      load_residual(e.group, e.counter);
    }
    if (kTmaRes && e.counter == 0) named_bar_sync(bar, 128);  // the barriers exist
    uint32_t next[8];
    if (e.group < nbox && !summed) {
      __syncwarp();
      tmem_ld_32x32b_x8(tacc + e.group * kCols, next);
    }
    for (int b = e.group; b < nbox; b += kGroups) {
      const int x = t.m0 + b * kCols;
      uint8_t* const dst = box + (e.counter % kBufs) * kBoxBytes;
      if (kTmaRes) {
        if (e.tid == 0 && b + kGroups < nbox) load_residual(b + kGroups, e.counter + 1);
        if (!mbar_wait_until(rbar + 8u * (e.counter % kBufs), (e.counter / kBufs) & 1,
                             globaltimer_ns() + kWaitLimitNs))
          atomicOr(p.c.status, kStatusTimeout);
      }
#pragma unroll 1
      for (int c = 0; c < kCols / 8; ++c) {
        const int col = x + c * 8;
        uint4 bq = make_uint4(0, 0, 0, 0), rq = bq;
        if (kEpi && p.bias && col < p.M) bq = __ldg(reinterpret_cast<const uint4*>(p.bias + col));
        if (has_r && col < p.M) {
          const size_t at = static_cast<size_t>(row) * p.M + col;
          if (in_bounds(p.c.status, at, 8, static_cast<size_t>(p.J) * p.M))
            rq = *reinterpret_cast<const uint4*>(p.residual + at);
        }
        if (summed)
          sum_parts(p, t, b * kCols + c * 8, e, next);
        else
          tmem_ld_wait();
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f32(next[j]);
        if (!summed) {
          const int nc = (c < kCols / 8 - 1 ? b : b + kGroups - 1) * kCols + c * 8 + 8;
          __syncwarp();
          if (nc < nbox * kCols) tmem_ld_32x32b_x8(tacc + nc, next);
        }
        uint4 z;
        if (kEpi) {
          if (p.bias) add8(v, bq);
          if (kKeepZ) z = pack8(v);
          with_act(p.act, [&](auto tag) { act8<decltype(tag)::value>(v); });
          // the residual's chunk lies where the result's will
          if (kTmaRes) add8(v, *chunk(dst, e.row, c));
          if (has_r) add8(v, rq);
        }
        const uint4 y = pack8(v);
        if (!kTmaRes && c == 0) {  // the box is free once its last store has been read
          if (e.tid == 0) tma_store_wait_read<0>();
          named_bar_sync(bar, 128);
        }
        *chunk(dst, e.row, c) = y;
        if (kKeepZ) *chunk(box + kBufs * kBoxBytes, e.row, c) = z;
      }
      fence_async_shared();
      named_bar_sync(bar, 128);
      if (e.tid == 0) {
        tma_store_2d(&p.tmOut, box_u32 + static_cast<uint32_t>(dst - box), x, y0);
        if (kKeepZ) tma_store_2d(&p.tmZ, box_u32 + kBufs * kBoxBytes, x, y0);
        tma_store_commit();
      }
      ++e.counter;
    }
  }
  static __device__ __forceinline__ void epilogue_drain(const Params&, EpiCtx& e) { store_drain(e); }
};

// Tensor map of a stored matrix of `rows` rows of `len` values, in boxes of 64 (or
// 32) values x box_rows rows, swizzled over the box's row.
bool encode_2d(CUtensorMap* tm, const void* base, int64_t len, int64_t rows, uint32_t box_rows,
               uint32_t box_cols = 64) {
  const uint64_t dims[2] = {static_cast<uint64_t>(len), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(len) * 2};
  const uint32_t box[2] = {box_cols, box_rows};
  return encode_tmap_bf16(tm, base, 2, dims, strides, box, static_cast<int>(box_cols * 2));
}

// How the tiles go over the pairs: where the last round has few tiles, each is
// split between several pairs. In nanoseconds: a step of a tile takes 310 and a
// tile's epilogue 1500 beside it, starting and ending 8500 for the forward with its
// activation, 7000 for dX, 4500 for dW, and joining s parts 3000 + 1600 s (their way
// through L2). dW of 12000 rows, 1280 -> 5120, 100 tiles on 74 pairs: 127 us in two
// rounds, 112 with the last 26 tiles split in two.
struct PairPlan {
  int split = 1;
  double ns = 0.0;
};
PairPlan plan_pairs(const LinearGemm& g, const DeviceInfo& dev) {
  const int64_t tiles =
      static_cast<int64_t>(ceil_div(g.J, 256)) * ceil_div(g.M, g.M > 128 ? 256 : 128);
  const int64_t steps = ceil_div(g.K, 64);
  const int64_t pairs = dev.sm_count / 2, rounds = tiles / pairs, tail = tiles % pairs;
  const double tile_ns = 310.0 * static_cast<double>(steps) + 1500.0;
  const double base = (g.b_mn ? 4500.0 : g.a_mn ? 7000.0 : 8500.0) +
                      static_cast<double>(rounds) * tile_ns;
  PairPlan best;
  best.ns = base + (tail > 0 ? tile_ns : 0.0);
  if (tail == 0) return best;
  for (int s = 2; s <= pairs / tail && s <= 16 && s * 4 <= steps; ++s) {
    const double ns =
        base + 310.0 * static_cast<double>((steps + s - 1) / s) + 4500.0 + 1600.0 * s;
    if (ns < best.ns) {
      best.ns = ns;
      best.split = s;
    }
  }
  return best;
}

template <bool kRowMn, bool kColMn, PairEpilogue kMode, bool kTail>
int launch_pair_as(const LinearGemm& g, int split, const DeviceInfo& dev, cudaStream_t s) {
  using Pol = DensePairPolicy<kRowMn, kColMn, kMode, kTail>;
  DensePairParams p;
  p.J = static_cast<int>(g.J);
  p.M = static_cast<int>(g.M);
  p.K = static_cast<int>(g.K);
  p.bn = g.M > 128 ? 256 : 128;
  p.tiles_m = ceil_div(g.M, p.bn);
  p.act = g.act;
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  // the row operand is B of the product (rows j), the column operand A (m)
  const bool ok =
      (kRowMn ? encode_2d(&p.tmRow, g.B, g.J, g.K, 64) : encode_2d(&p.tmRow, g.B, g.K, g.J, 128)) &&
      (kColMn ? encode_2d(&p.tmCol, g.A, g.M, g.K, 64)
              : encode_2d(&p.tmCol, g.A, g.K, g.M, static_cast<uint32_t>(p.bn / 2))) &&
      encode_2d(&p.tmOut, g.Out, g.M, g.J, 128, Pol::kCols) &&
      encode_2d(&p.tmZ, kMode == kForwardZ ? g.Z : kMode == kForwardResidual ? g.residual : g.Out,
                g.M, g.J, 128, Pol::kCols);
  if (!ok) return -2;
  const int64_t tiles = static_cast<int64_t>(ceil_div(g.J, 256)) * p.tiles_m;
  if (tiles > 0x7fffffff) return -2;
  p.split = split;
  p.tail = split > 1 ? static_cast<int>(tiles % (dev.sm_count / 2)) : 0;
  p.whole = static_cast<int>(tiles) - p.tail;
  p.ws = g.ws;
  p.counters = g.counters;
  const uint32_t smem =
      setup_common<Pol>(p.c, p.whole + p.tail * p.split, 128 * 128, (p.bn / 2) * 128, p.bn, kRowMn,
                        kColMn, g.status, dev);
  if (!smem) return -3;
  p.c.idesc = idesc_bf16(256, p.bn, kRowMn, kColMn);
  return launch_gemm_pair<Pol>(p, smem, dev, s, true);
}

template <bool kRowMn, bool kColMn, PairEpilogue kMode>
int launch_pair(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s) {
  const int split = plan_pairs(g, dev).split;
  return split > 1 ? launch_pair_as<kRowMn, kColMn, kMode, true>(g, split, dev, s)
                   : launch_pair_as<kRowMn, kColMn, kMode, false>(g, 1, dev, s);
}

// --------------------------------------------------------------- clusters ----
// The same products where the 256 x 256 tiles are few or mostly empty
// (split_kernel of stream_gemm.cuh): a tile is 128 columns m of the output (A's
// rows) x nb rows j, its steps shared by a cluster of cs CTAs.
struct DenseSplitParams {
  StreamCommon c;
  CUtensorMap tmA, tmB;
  int M, J, K, tiles_j;
  int act;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;  // may be Out
  __nv_bfloat16* Out;
  __nv_bfloat16* Z;
};

template <bool kAMn, bool kBMn, bool kEpi>
struct DenseSplitPolicy {
  using Params = DenseSplitParams;
  static constexpr uint32_t kSmemBytes = 0;
  static constexpr uint64_t kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;

  static __device__ __forceinline__ void prefetch(const Params& p) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  static __device__ __forceinline__ int steps(const Params& p) { return ceil_div_dev(p.K, 64); }
  // tiles of the same rows of A are neighbours: they share A through L2
  static __device__ __forceinline__ int m_of(const Params& p, int tile) {
    return tile / p.tiles_j * 128;
  }
  static __device__ __forceinline__ int j_of(const Params& p, int tile) {
    return tile % p.tiles_j * p.c.nb;
  }
  static __device__ __forceinline__ void load_a(const Params& p, int tile, int k, uint32_t dst,
                                                uint32_t bar) {
    const int m = m_of(p, tile);
    if (kAMn) {
      tma_load_2d(dst, &p.tmA, bar, m, k * 64);
      tma_load_2d(dst + 8192u, &p.tmA, bar, m + 64, k * 64);
    } else {
      tma_load_2d(dst, &p.tmA, bar, k * 64, m);
    }
  }
  static __device__ __forceinline__ void load_b(const Params& p, int tile, int k, uint32_t dst,
                                                uint32_t bar) {
    const int j = j_of(p, tile);
    if (kBMn) {
      for (int q = 0; q < p.c.nb; q += 64)
        tma_load_2d(dst + static_cast<uint32_t>(q) * 128u, &p.tmB, bar, j + q, k * 64);
    } else {
      tma_load_2d(dst, &p.tmB, bar, k * 64, j);
    }
  }
  static __device__ __forceinline__ uint64_t adesc(uint32_t a) {
    return kAMn ? mnmajor_desc(a, 0) : kmajor_desc(a, 0);
  }
  static __device__ __forceinline__ uint64_t bdesc(uint32_t b) {
    return kBMn ? mnmajor_desc(b, 0) : kmajor_desc(b, 0);
  }
  static __device__ __forceinline__ int columns(const Params& p, int tile) {
    return min(p.c.nb, p.J - j_of(p, tile));
  }
  static __device__ __forceinline__ void finish8(const Params& p, int tile, int octet, int col,
                                                 float (&v)[8]) {
    const int j = j_of(p, tile) + col, m = m_of(p, tile) + octet * 8;
    const size_t at = static_cast<size_t>(j) * p.M + m;
    if (m >= p.M || !in_bounds(p.c.status, at, 8, static_cast<size_t>(p.J) * p.M)) return;
    uint4 r = make_uint4(0, 0, 0, 0);
    if (kEpi) {
      if (p.residual) r = *reinterpret_cast<const uint4*>(p.residual + at);
      if (p.bias) add8(v, __ldg(reinterpret_cast<const uint4*>(p.bias + m)));
      if (p.Z) *reinterpret_cast<uint4*>(p.Z + at) = pack8(v);
      with_act(p.act, [&](auto tag) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_f<decltype(tag)::value, true>(v[i]);
      });
      if (p.residual) add8(v, r);
    }
    *reinterpret_cast<uint4*>(p.Out + at) = pack8(v);
  }
};

struct SplitChoice {
  int nb = 0;  // columns of a tile; 0: CTA pairs
  int cs = 1;  // CTAs per tile
};

template <bool kAMn, bool kBMn, bool kEpi>
int launch_split(const LinearGemm& g, SplitChoice ch, const DeviceInfo& dev, cudaStream_t s) {
  using Pol = DenseSplitPolicy<kAMn, kBMn, kEpi>;
  DenseSplitParams p;
  p.M = static_cast<int>(g.M);
  p.J = static_cast<int>(g.J);
  p.K = static_cast<int>(g.K);
  p.tiles_j = ceil_div(g.J, ch.nb);
  p.act = g.act;
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  p.Out = static_cast<__nv_bfloat16*>(g.Out);
  p.Z = static_cast<__nv_bfloat16*>(g.Z);
  if (!(kAMn ? encode_2d(&p.tmA, g.A, g.M, g.K, 64) : encode_2d(&p.tmA, g.A, g.K, g.M, 128)) ||
      !(kBMn ? encode_2d(&p.tmB, g.B, g.J, g.K, 64)
             : encode_2d(&p.tmB, g.B, g.K, g.J, static_cast<uint32_t>(ch.nb))))
    return -2;
  const uint32_t smem =
      stream_setup<Pol>(p.c, ch.nb, kAMn, kBMn, nullptr, nullptr, g.status, g.wait_ns, dev);
  if (!smem) return -3;
  return split_launch<Pol>(p, ceil_div(g.M, 128) * p.tiles_j, ch.cs, smem, dev, s);
}

// Clusters of cs CTAs (one CTA per SM) that run at once: a cluster stays within
// a group of SMs, whose count no cluster size above 2 divides evenly.
int resident_clusters(int cs, const DeviceInfo& dev) {
  static std::atomic<int> known[kMaxDevices][9];
  if (cs == 1) return dev.sm_count;
  if (dev.device < 0 || dev.device >= kMaxDevices) return dev.sm_count / 8;
  int n = known[dev.device][cs].load();
  if (n == 0) {
    n = split_resident<DenseSplitPolicy<false, false, true>>(cs, dev);
    known[dev.device][cs].store(n);  // (0: asked again)
  }
  return n > 0 ? n : std::max(1, dev.sm_count / (2 * cs));
}

// CTA pairs or clusters, by a model of both in nanoseconds (plan_pairs; below), a
// least-squares fit over the forward, dX and dW of nine shapes from 104 -> 96 to 4096
// -> 14336 at 1 to 3000 rows with cold weights. Over those its choice is 1% slower
// than the fastest on average, 21% at worst (700 rows through 512 -> 2048, 13.1 us for
// 10.8). Of choices that the model holds equal (under weights_ns, the weights' read)
// the first, of fewest columns and CTAs, is taken: for one token through 4096 -> 14336
// a CTA for each of the 112 tiles, 24.1 us; the fastest is 24.3. The pairs' side has
// no such term: for sums far longer than those of the fit it may choose them wrongly.
// 64 rows through 1024 -> 1024: 6.9 us in
// clusters of 4, 15.3 on pairs; 450 rows through 4096 -> 14336: 56 on pairs, 105 in
// clusters.
SplitChoice choose_split(const LinearGemm& g, const DeviceInfo& dev) {
  const int64_t ks = ceil_div(g.K, 64), tm = ceil_div(g.M, 128);
  const double weights_ns = 2.0 * static_cast<double>(g.M) * static_cast<double>(g.K) / 5200.0;
  SplitChoice best;
  double best_ns = plan_pairs(g, dev).ns;
  const int64_t most = std::min<int64_t>(kStreamMaxNb, (g.J + 15) / 16 * 16);
  const int unit = g.b_mn ? 64 : 16;  // an MN-major operand comes in whole boxes of 64
  for (int nb = unit; nb <= std::max<int64_t>(most, unit); nb += unit) {
    const int64_t tiles = tm * ceil_div(g.J, nb);
    if (tiles > 4 * dev.sm_count) continue;
    const double n = static_cast<double>(std::min<int64_t>(nb, g.J));
    for (int cs : {1, 2, 3, 4, 6, 8}) {
      if (cs > ks) break;
      const int resident = resident_clusters(cs, dev);
      const double waves = static_cast<double>((tiles + resident - 1) / resident);
      const double cta_ns = 227.0 * static_cast<double>((ks + cs - 1) / cs) - 48.0 * n +
                            109.0 * n / cs + (cs > 1 ? (147.0 + 14.4 * n) * cs - 673.0 : 0.0);
      const double ns = 5550.0 + std::max(waves * cta_ns + (waves - 1.0) * 4000.0, weights_ns);
      if (ns < best_ns) {
        best_ns = ns;
        best.nb = nb;
        best.cs = cs;
      }
    }
  }
  return best;
}

}  // namespace

size_t linear_ws_bytes(const DeviceInfo& dev) {  // a part of 256 x 256 per pair
  return static_cast<size_t>(dev.sm_count / 2) * 256 * 256 * sizeof(float);
}
int linear_counters(const DeviceInfo& dev) { return dev.sm_count; }

int launch_linear_umma(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s) {
  const SplitChoice ch = choose_split(g, dev);

  if (g.a_mn && g.b_mn)
    return ch.nb ? launch_split<true, true, false>(g, ch, dev, s)
                 : launch_pair<true, true, kPlain>(g, dev, s);
  if (g.a_mn)
    return ch.nb ? launch_split<true, false, false>(g, ch, dev, s)
                 : launch_pair<false, true, kPlain>(g, dev, s);
  if (ch.nb) return launch_split<false, false, true>(g, ch, dev, s);
  if (g.Z) return launch_pair<false, false, kForwardZ>(g, dev, s);
  return g.residual ? launch_pair<false, false, kForwardResidual>(g, dev, s)
                    : launch_pair<false, false, kForward>(g, dev, s);
}

}  // namespace dyra
