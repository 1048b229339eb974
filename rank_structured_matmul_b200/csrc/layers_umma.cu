// layers_umma.cu - the bf16 products of the dense layer on tcgen05 tensor
// cores: fp32 accumulation in tensor memory, operands by TMA, the epilogue
// (bias, activation, residual, the kept pre-activations) on the accumulator.
#include <algorithm>

#include "layers.h"
#include "layers_math.cuh"
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
      for (int i = 0; i < 64; ++i) v[i] = act_f<ACT>(v[i]);
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

}  // namespace

int launch_linear_umma(const LinearGemm& g, const DeviceInfo& dev, cudaStream_t s, bool pdl) {
  if (g.a_mn && g.b_mn) return launch_pair<true, true, false>(g, dev, s, pdl);
  if (g.a_mn) return launch_pair<false, true, false>(g, dev, s, pdl);
  return launch_pair<false, false, true>(g, dev, s, pdl);
}

}  // namespace dyra
