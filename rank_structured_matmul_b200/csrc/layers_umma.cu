// layers_umma.cu - the bf16 products of the dense layer on tcgen05 tensor
// cores: fp32 accumulation in tensor memory, operands by TMA, the epilogue
// (bias, activation, residual, the kept pre-activations) on the accumulator.
#include <algorithm>

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

// ------------------------------------------------------------ CTA pairs ----
// Out tile of 256 rows (j) x bn columns (m) on a CTA pair: CTA r loads rows
// j0 + 128 r of the row operand and columns m0 + (bn / 2) r of the other, each
// K-major (one box of 64 k) or MN-major (boxes of 64 x 64 k).
struct DensePairParams {
  GemmCommon c;
  CUtensorMap tmRow;  // row operand (J x K, or K x J when MN-major)
  CUtensorMap tmCol;  // column operand (M x K, or K x M when MN-major)
  CUtensorMap tmOut;  // J x M, box (64, 128), store
  CUtensorMap tmZ;    // the same over the kept pre-activations
  int J, M, K, bn, tiles_m;
  int act, keep_z;
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
};

// kEpi compiles the forward's epilogue in; the gradients' products store the
// accumulator as it is.
template <bool kRowMn, bool kColMn, bool kEpi>
struct DensePairPolicy {
  using Params = DensePairParams;
  struct Tile {
    int j0, m0;
  };
  static constexpr uint32_t kEpiSmemBytes = kStoreBoxes * kStoreBoxBytes;

  static __device__ __forceinline__ void prefetch(const Params& p) {
    tma_prefetch_desc(&p.tmRow);
    tma_prefetch_desc(&p.tmCol);
    tma_prefetch_desc(&p.tmOut);
  }
  static __device__ __forceinline__ void decode(const Params& p, int tile, Tile& t) {
    t.j0 = (tile / p.tiles_m) * 256;
    t.m0 = (tile % p.tiles_m) * p.bn;
  }
  static __device__ __forceinline__ int kiters(const Params& p, const Tile&) {
    return ceil_div_dev(p.K, 64);
  }
  static __device__ __forceinline__ void load(const Params& p, const Tile& t, int it, uint32_t sa,
                                              uint32_t sb, uint32_t bar, uint32_t rank) {
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
  static __device__ __forceinline__ int ksteps(const Params& p, const Tile&, int it) {
    return min(4, ceil_div_dev(p.K - it * 64, 16));
  }
  static __device__ __forceinline__ uint64_t adesc(const Params&, uint32_t a, int ks) {
    return kRowMn ? mnmajor_desc(a, ks) : kmajor_desc(a, ks);
  }
  static __device__ __forceinline__ uint64_t bdesc(const Params&, uint32_t b, int ks) {
    return kColMn ? mnmajor_desc(b, ks) : kmajor_desc(b, ks);
  }

  // Sixty-four values of this thread's row as bf16 into the next store box and
  // out: as store_box_bf16, from registers.
  static __device__ __forceinline__ void emit(const float (&v)[64], const CUtensorMap* tm, int x,
                                              int y, EpiCtx& e) {
    const uint32_t buf = e.counter % kStoreBoxes;
    ++e.counter;
    if (e.tid == 0) tma_store_wait_read<kStoreBoxes - 1>();
    named_bar_sync(1, 128);
    uint8_t* sbuf = e.smem + buf * kStoreBoxBytes;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint4 q;
      q.x = pack_bf16x2(v[8 * c], v[8 * c + 1]);
      q.y = pack_bf16x2(v[8 * c + 2], v[8 * c + 3]);
      q.z = pack_bf16x2(v[8 * c + 4], v[8 * c + 5]);
      q.w = pack_bf16x2(v[8 * c + 6], v[8 * c + 7]);
      *reinterpret_cast<uint4*>(sbuf + e.row * 128 + ((c ^ (e.row & 7)) * 16)) = q;
    }
    fence_async_shared();
    named_bar_sync(1, 128);
    if (e.tid == 0) {
      tma_store_2d(tm, e.smem_u32 + buf * kStoreBoxBytes, x, y);
      tma_store_commit();
    }
  }
  static __device__ __forceinline__ void add8(float* v, const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] += __uint_as_float(w[j] << 16);
      v[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void epilogue(const Params& p, const Tile& t, uint32_t tacc,
                                                  EpiCtx& e) {
    const int y0 = t.j0 + 128 * e.rank;
    if constexpr (!kEpi) {
      for (int bx = 0; bx < p.bn / 64 && t.m0 + bx * 64 < p.M; ++bx)
        store_box_bf16(tacc, bx * 64, &p.tmOut, t.m0 + bx * 64, y0, e);
    } else {
      with_act(p.act, [&](auto tag) { boxes<decltype(tag)::value>(p, t, tacc, e, y0); });
    }
  }
  template <int ACT>
  static __device__ __forceinline__ void boxes(const Params& p, const Tile& t, uint32_t tacc,
                                               EpiCtx& e, int y0) {
    const int row = y0 + e.row;
    for (int bx = 0; bx < p.bn / 64; ++bx) {
      const int x = t.m0 + bx * 64;
      if (x >= p.M) break;
      // the row's residual and the bias first: their latency passes during the
      // loads from tensor memory (8 columns per load, all inside or all beyond M)
      uint4 rq[8], bq[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const bool in = x + c * 8 < p.M;
        const size_t at = static_cast<size_t>(row) * p.M + x + c * 8;
        rq[c] = make_uint4(0, 0, 0, 0);
        if (p.residual && in && row < p.J &&
            in_bounds(p.c.status, at, 8, static_cast<size_t>(p.J) * p.M))
          rq[c] = *reinterpret_cast<const uint4*>(p.residual + at);
        bq[c] = p.bias && in ? __ldg(reinterpret_cast<const uint4*>(p.bias + x + c * 8))
                             : make_uint4(0, 0, 0, 0);
      }
      uint32_t raw[2][32];
      tmem_ld_32x32b_x32(tacc + bx * 64, raw[0]);
      tmem_ld_32x32b_x32(tacc + bx * 64 + 32, raw[1]);
      tmem_ld_wait();
      float v[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = f32(raw[i / 32][i % 32]);
      if (p.bias) {
#pragma unroll
        for (int c = 0; c < 8; ++c) add8(v + 8 * c, bq[c]);
      }
      if (p.keep_z) emit(v, &p.tmZ, x, y0, e);
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = act_f<ACT, true>(v[i]);
      if (p.residual) {
#pragma unroll
        for (int c = 0; c < 8; ++c) add8(v + 8 * c, rq[c]);
      }
      emit(v, &p.tmOut, x, y0, e);
    }
  }
  static __device__ __forceinline__ void epilogue_drain(const Params&, EpiCtx& e) { store_drain(e); }
};

// Tensor map of a stored matrix of `rows` rows of `len` values, in boxes of 64
// values x box_rows rows.
bool encode_2d(CUtensorMap* tm, const void* base, int64_t len, int64_t rows, uint32_t box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(len), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(len) * 2};
  const uint32_t box[2] = {64, box_rows};
  return encode_tmap_bf16(tm, base, 2, dims, strides, box, 128);
}

template <bool kRowMn, bool kColMn, bool kEpi>
int launch_pair(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s, bool pdl) {
  using Pol = DensePairPolicy<kRowMn, kColMn, kEpi>;
  DensePairParams p;
  p.J = static_cast<int>(g.J);
  p.M = static_cast<int>(g.M);
  p.K = static_cast<int>(g.K);
  p.bn = g.M > 128 ? 256 : 128;
  p.tiles_m = ceil_div(g.M, p.bn);
  p.act = g.act;
  p.keep_z = g.Z != nullptr ? 1 : 0;
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  // the row operand is B of the product (rows j), the column operand A (m)
  const bool ok =
      (kRowMn ? encode_2d(&p.tmRow, g.B, g.J, g.K, 64) : encode_2d(&p.tmRow, g.B, g.K, g.J, 128)) &&
      (kColMn ? encode_2d(&p.tmCol, g.A, g.M, g.K, 64)
              : encode_2d(&p.tmCol, g.A, g.K, g.M, static_cast<uint32_t>(p.bn / 2))) &&
      encode_2d(&p.tmOut, g.Out, g.M, g.J, 128) &&
      encode_2d(&p.tmZ, g.Z ? g.Z : g.Out, g.M, g.J, 128);
  if (!ok) return -2;
  const int64_t tiles = static_cast<int64_t>(ceil_div(g.J, 256)) * p.tiles_m;
  if (tiles > 0x7fffffff) return -2;
  const uint32_t smem =
      setup_common<Pol>(p.c, static_cast<int>(tiles), 128 * 128, (p.bn / 2) * 128, p.bn, kRowMn,
                        kColMn, g.status, dev);
  if (!smem) return -3;
  p.c.idesc = idesc_bf16(256, p.bn, kRowMn, kColMn);
  return launch_gemm_pair<Pol>(p, smem, dev, s, pdl);
}

// ---------------------------------------------------------------- streams ----
// The same products where the 256 x 256 tiles are few (stream_gemm.cuh): a tile
// is 128 columns m of the output (A's rows) x nb rows j, so a thread holds one m
// and a warp's stores of one j are 64 contiguous bytes.
struct DenseStreamParams {
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
struct DenseStreamPolicy {
  using Params = DenseStreamParams;
  struct Acc {};
  static constexpr uint32_t kSmemBytes = 0;
  static constexpr uint64_t kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;

  static __device__ __forceinline__ void prefetch(const Params& p) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
  }
  static __device__ __forceinline__ void setup(const Params&, uint8_t*) {}
  static __device__ __forceinline__ void shape(const Params& p, uint8_t*, int& tiles, int& nsub,
                                               int& ks) {
    tiles = ceil_div_dev(p.M, 128) * p.tiles_j;
    nsub = 1;
    ks = ceil_div_dev(p.K, 64);
  }
  // tiles of the same rows of A are neighbours: they share A through L2
  static __device__ __forceinline__ int m_of(const Params& p, int tile) {
    return tile / p.tiles_j * 128;
  }
  static __device__ __forceinline__ int j_of(const Params& p, int tile) {
    return tile % p.tiles_j * p.c.nb;
  }
  static __device__ __forceinline__ void load_a(const Params& p, uint8_t*, int tile, int, int k,
                                                uint32_t dst, uint32_t bar) {
    const int m = m_of(p, tile);
    if (kAMn) {
      tma_load_2d(dst, &p.tmA, bar, m, k * 64);
      tma_load_2d(dst + 8192u, &p.tmA, bar, m + 64, k * 64);
    } else {
      tma_load_2d(dst, &p.tmA, bar, k * 64, m);
    }
  }
  static __device__ __forceinline__ void load_b(const Params& p, uint8_t*, int tile, int, int k,
                                                uint32_t dst, uint32_t bar) {
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
  // Columns col0 .. col0 + n - 1 of the tile, this thread's row: out.
  template <int ACT>
  static __device__ __forceinline__ void finish(const Params& p, int j0, int m, float bias,
                                                const float (&v)[32], int n) {
    if (m >= p.M) return;
    const size_t extent = static_cast<size_t>(p.J) * p.M;
    float r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const size_t at = static_cast<size_t>(j0 + i) * p.M + m;
      r[i] = kEpi && p.residual && i < n && in_bounds(p.c.status, at, 1, extent)
                 ? __bfloat162float(p.residual[at])
                 : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i >= n) break;
      const size_t at = static_cast<size_t>(j0 + i) * p.M + m;
      if (!in_bounds(p.c.status, at, 1, extent)) continue;
      const float z = v[i] + bias;
      if (kEpi && p.Z) p.Z[at] = __float2bfloat16_rn(z);
      p.Out[at] = __float2bfloat16_rn(act_f<ACT, true>(z) + r[i]);
    }
  }
  template <class Release>
  static __device__ __forceinline__ void segment(const Params& p, uint8_t*, const StreamSeg& s,
                                                 int per_tile, uint32_t tacc, StreamEpi& e, Acc&,
                                                 const Release& release) {
    const int j0 = j_of(p, s.tile), m = m_of(p, s.tile) + e.row;
    const int n = min(p.c.nb, p.J - j0);
    const float bias = kEpi && p.bias && m < p.M ? __bfloat162float(p.bias[m]) : 0.f;
    auto out = [&](const float(&v)[32], int col) {
      if (kEpi)
        with_act(p.act, [&](auto tag) {
          finish<decltype(tag)::value>(p, j0 + col, m, bias, v, n - col);
        });
      else
        finish<DYRA_ACT_NONE>(p, j0 + col, m, bias, v, n - col);
    };
    float* part = stream_part(p.c, static_cast<int>(blockIdx.x), s.first) + e.row;
    for (int col = 0; col < n; col += 32) {
      __syncwarp();
      uint32_t raw[32];
      tmem_ld_32x32b_x32(tacc + col, raw);
      tmem_ld_wait();
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = f32(raw[i]);
      if (s.whole) {
        out(v, col);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i < n) part[(col + i) * 128] = v[i];
      }
    }
    release();
    if (s.whole) return;
    int c0, c1;
    if (!stream_arrive(p.c, s, per_tile, e, c0, c1)) return;
    for (int col = 0; col < n; col += 32) {
      float v[32];
      stream_sum(p.c, c0, c1, e.row, col, n - col, v);
      out(v, col);
    }
  }
  static __device__ __forceinline__ void nothing(const Params&, const StreamEpi&) {}
};

template <bool kAMn, bool kBMn, bool kEpi>
int launch_stream(const LinearGemm& g, int nb, const DeviceInfo& dev, cudaStream_t s, bool pdl) {
  using Pol = DenseStreamPolicy<kAMn, kBMn, kEpi>;
  DenseStreamParams p;
  p.M = static_cast<int>(g.M);
  p.J = static_cast<int>(g.J);
  p.K = static_cast<int>(g.K);
  p.tiles_j = ceil_div(g.J, nb);
  p.act = g.act;
  p.bias = static_cast<const __nv_bfloat16*>(g.bias);
  p.residual = static_cast<const __nv_bfloat16*>(g.residual);
  p.Out = static_cast<__nv_bfloat16*>(g.Out);
  p.Z = static_cast<__nv_bfloat16*>(g.Z);
  if (!(kAMn ? encode_2d(&p.tmA, g.A, g.M, g.K, 64) : encode_2d(&p.tmA, g.A, g.K, g.M, 128)) ||
      !(kBMn ? encode_2d(&p.tmB, g.B, g.J, g.K, 64)
             : encode_2d(&p.tmB, g.B, g.K, g.J, static_cast<uint32_t>(nb))))
    return -2;
  const uint32_t smem =
      stream_setup<Pol>(p.c, nb, kAMn, kBMn, g.ws, g.counters, g.status, dev);
  if (!smem) return -3;
  return stream_launch<Pol>(p, smem, dev, s, pdl);
}

// Columns of a stream tile for the product, 0: the CTA pairs take it.
int stream_columns(const LinearGemm& g, const DeviceInfo& dev) {
  const int64_t pair_tiles =
      static_cast<int64_t>(ceil_div(g.J, 256)) * ceil_div(g.M, g.M > 128 ? 256 : 128);
  if (g.J > kStreamMaxNb && pair_tiles > dev.sm_count / 2) return 0;
  const int tj = ceil_div(g.J, kStreamMaxNb);
  int nb = ceil_div(ceil_div(g.J, tj), 16) * 16;
  if (g.b_mn) nb = nb <= 64 ? 64 : 128;  // whole boxes of 64
  // steps are counted in 32 bits
  if (static_cast<double>(ceil_div(g.M, 128)) * ceil_div(g.J, nb) * ceil_div(g.K, 64) > 1e9)
    return 0;
  return nb;
}

}  // namespace

size_t linear_ws_bytes(const DeviceInfo& dev) {
  return static_cast<size_t>(dev.sm_count) * 2 * kStreamMaxNb * 128 * sizeof(float);
}

// Tiles of a stream: one per 128 columns m of up to kStreamMaxNb rows, or where
// the pairs' tiles are at most half the SMs, four of 128 x 128 for each of those.
int linear_counters(int d_in, int d_out, const DeviceInfo& dev) {
  return std::max(ceil_div(std::max(d_in, d_out), 128), dev.sm_count / 2 * 4);
}

int launch_linear_umma(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s, bool pdl) {
  const int nb = stream_columns(g, dev);
  if (g.a_mn && g.b_mn)
    return nb ? launch_stream<true, true, false>(g, nb, dev, s, pdl)
              : launch_pair<true, true, false>(g, dev, s, pdl);
  if (g.a_mn)
    return nb ? launch_stream<true, false, false>(g, nb, dev, s, pdl)
              : launch_pair<false, true, false>(g, dev, s, pdl);
  return nb ? launch_stream<false, false, true>(g, nb, dev, s, pdl)
            : launch_pair<false, false, true>(g, dev, s, pdl);
}

}  // namespace dyra
