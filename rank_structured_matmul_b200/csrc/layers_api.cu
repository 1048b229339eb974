// layers_api.cu - the C ABI declared in include/dyra_layers.h: handles,
// argument checks, and the choice between the tensor-core kernels (bf16) and
// the CUDA-core ones (fp32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <new>

#include "api_util.h"
#include "dyra_debug.h"
#include "layers.h"

using namespace dyra;

struct dyra_dense {
  int d_in = 0, d_out = 0;
  dyra_dtype_t dtype = DYRA_BF16;
  DeviceInfo dev;
  bool simt = false;        // fp32, or DYRA_KERNELS=simt (debugging)
  float* colsum = nullptr;  // kColSumChunks x d_out partial column sums
  int* counters = nullptr;  // col_sum_blocks(d_out) arrival counters, zero between calls
  float* ws = nullptr;      // tensor cores: parts of split tiles, and
  int* tiles = nullptr;     // their arrival counters, zero between calls
  int n_tiles = 0;
  int* status = nullptr;
  void* base = nullptr;     // the one allocation that holds them
  size_t bytes = 0;
  unsigned long long wait_ns = 0;  // diagnostic wait limit (0: the default)
};

struct dyra_moe {
  MoeShape m = {};
  dyra_dtype_t dtype = DYRA_BF16;
  DeviceInfo dev;
  bool simt = false;
  void* hidden = nullptr;  // the hidden values of one group of kMoeTokens tokens
  float* part = nullptr;   // CUDA cores: its slots' outputs; tensor cores: parts of split tiles
  double* logits = nullptr;  // the router's
  int* tiles = nullptr;    // arrival counters, zero between calls: the router's, then the tiles'
  int* status = nullptr;
  void* base = nullptr;    // the one allocation that holds them
  size_t bytes = 0;
  int n_tiles = 0;
  unsigned long long wait_ns = 0;  // as above
};

namespace {

// of rows and widths: tile origins up to 511 beyond the last stay inside 32-bit coordinates
constexpr int64_t kMaxRows = (static_cast<int64_t>(1) << 31) - 512;

bool simt_requested() {
  const char* kv = std::getenv("DYRA_KERNELS");
  return kv != nullptr && std::strcmp(kv, "simt") == 0;
}

bool known_act(int act) { return act >= DYRA_ACT_NONE && act <= DYRA_ACT_SILU; }

// The bytes of an argument; a NULL one has none.
struct Span {
  uintptr_t at;
  size_t bytes;
  Span(const void* p, size_t n) : at(reinterpret_cast<uintptr_t>(p)), bytes(p ? n : 0) {}
  bool meets(const Span& o) const {
    return bytes && o.bytes && at < o.at + o.bytes && o.at < at + bytes;
  }
  // the same array, or no byte in common
  bool same_or_apart(const Span& o) const { return at == o.at || !meets(o); }
};
bool meets_any(const Span& a, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (a.meets(o)) return true;
  return false;
}

// A handle's buffers are parts of one allocation (a bf16 dense handle takes 0.05 ms to
// make, with an allocation per buffer 0.13). Those that begin at zero come first.
struct Layout {
  size_t total = 0;
  size_t add(size_t bytes) {
    const size_t at = total;
    total += (bytes + 255) & ~static_cast<size_t>(255);
    return at;
  }
};
template <class T>
T* part_at(void* base, size_t at) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + at);
}
int allocate(void** base, const Layout& l, size_t zeroed) {
  const int rc = dev_alloc(base, l.total);
  if (rc) return rc;
  // done before any stream can use the handle
  if (cudaMemset(*base, 0, zeroed) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
    cudaGetLastError();
    dev_free(*base);
    return DYRA_ERR_CUDA;
  }
  return DYRA_OK;
}

// A call that gave up may leave arrival counters behind: they start again.
int read_status(const DeviceInfo& dev, int* status, int* tiles, int n_tiles) {
  DeviceGuard g(dev.device);
  if (!g.ok || cudaDeviceSynchronize() != cudaSuccess) return DYRA_ERR_CUDA;
  int st = 0;
  if (cudaMemcpy(&st, status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(status, 0, sizeof(int)) != cudaSuccess ||
      (st != 0 && n_tiles && cudaMemset(tiles, 0, sizeof(int) * n_tiles) != cudaSuccess) ||
      cudaStreamSynchronize(nullptr) != cudaSuccess)
    return DYRA_ERR_CUDA;
  return st;
}

int launched(int rc) {
  if (rc == 0) return DYRA_OK;
  cudaGetLastError();
  return DYRA_ERR_CUDA;
}

int linear(const dyra_dense* p, const LinearGemm& g, cudaStream_t s) {
  if (p->dtype == DYRA_F32) return launch_linear_f32(g, p->dev, s);
  if (p->simt) return launch_linear_simt(g, p->dev, s);
  return launch_linear_umma(g, p->dev, s);
}

template <class T>
int act_backward(const dyra_dense* p, const void* dY, const void* Z, int act, void* dZ,
                 void* dbias, int64_t N, cudaStream_t s) {
  return launch_act_backward<T>(static_cast<const T*>(dY), static_cast<const T*>(Z), act,
                                static_cast<T*>(dZ), static_cast<T*>(dbias), N, p->d_out,
                                p->colsum, p->counters, p->status, p->dev, s);
}

template <class T>
int moe_route(const dyra_moe* p, const void* X, const void* Wr, int32_t* ids, float* weights,
              int64_t N, cudaStream_t s) {
  return launch_moe_route<T>(p->m, static_cast<const T*>(X), static_cast<const T*>(Wr), ids,
                             weights, N, p->logits, p->tiles, s);
}

template <class T>
int moe_experts(const dyra_moe* p, const void* X, const int32_t* ids, const float* weights,
                const void* Wgu, const void* Wd, const void* residual, void* Y, int n, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (!p->simt)
      return launch_moe_experts_umma(p->m, static_cast<const T*>(X), ids, weights,
                                     static_cast<const T*>(Wgu), static_cast<const T*>(Wd),
                                     static_cast<const T*>(residual), static_cast<T*>(Y), n,
                                     static_cast<T*>(p->hidden), p->part,
                                     p->tiles + moe_route_counters(), p->status, p->wait_ns, p->dev, s);
  return launch_moe_experts_simt<T>(p->m, static_cast<const T*>(X), ids, weights,
                                    static_cast<const T*>(Wgu), static_cast<const T*>(Wd),
                                    static_cast<const T*>(residual), static_cast<T*>(Y), n,
                                    static_cast<T*>(p->hidden), p->part, p->status, p->dev, s);
}

// What the calls on N tokens are given.
Span rows_of(const dyra_moe* p, const void* a, int64_t N) {
  return Span(a, elem_size(p->dtype) * N * p->m.d);
}
Span slots_of(const dyra_moe* p, const void* a, int64_t N) {  // ids and weights
  return Span(a, static_cast<size_t>(4) * N * p->m.top_k);
}
Span router_of(const dyra_moe* p, const void* Wr) {
  return Span(Wr, elem_size(p->dtype) * p->m.experts * p->m.d);
}
// `halves` 2: gate and up, 1: down
Span experts_of(const dyra_moe* p, const void* w, int halves) {
  return Span(w, elem_size(p->dtype) * p->m.experts * halves * p->m.d * p->m.f);
}

// The shared checks of the calls on N tokens: DYRA_OK to go on.
int moe_check(const dyra_moe* p, int64_t N) {
  if (p == nullptr || N < 0 || N > kMaxRows) return DYRA_ERR_INVALID_ARG;
  return DYRA_OK;
}

int run_experts(const dyra_moe* p, const void* X, const int32_t* ids, const float* weights,
                const void* Wgu, const void* Wd, const void* residual, void* Y, int64_t N,
                cudaStream_t s) {
  int rc = moe_check(p, N);
  if (rc || N == 0) return rc;
  if (X == nullptr || ids == nullptr || weights == nullptr || Wgu == nullptr || Wd == nullptr ||
      Y == nullptr)
    return DYRA_ERR_INVALID_ARG;
  for (const void* q : {X, static_cast<const void*>(ids), static_cast<const void*>(weights), Wgu,
                        Wd, residual, static_cast<const void*>(Y)})
    if (!aligned16(q)) return DYRA_ERR_ALIGNMENT;
  const Span y = rows_of(p, Y, N);
  if (meets_any(y, {rows_of(p, X, N), slots_of(p, ids, N), slots_of(p, weights, N),
                    experts_of(p, Wgu, 2), experts_of(p, Wd, 1)}) ||
      !y.same_or_apart(rows_of(p, residual, N)))
    return DYRA_ERR_INVALID_ARG;
  DeviceGuard g(p->dev.device);
  if (!g.ok) return DYRA_ERR_CUDA;
  const size_t row = elem_size(p->dtype) * p->m.d;
  for (int64_t n0 = 0; n0 < N && rc == 0; n0 += kMoeTokens) {
    const int n = static_cast<int>(std::min<int64_t>(kMoeTokens, N - n0));
    const void* x = static_cast<const char*>(X) + n0 * row;
    const void* r = residual ? static_cast<const char*>(residual) + n0 * row : nullptr;
    void* y = static_cast<char*>(Y) + n0 * row;
    rc = p->dtype == DYRA_F32
             ? moe_experts<float>(p, x, ids + n0 * p->m.top_k, weights + n0 * p->m.top_k, Wgu, Wd,
                                  r, y, n, s)
             : moe_experts<__nv_bfloat16>(p, x, ids + n0 * p->m.top_k, weights + n0 * p->m.top_k,
                                          Wgu, Wd, r, y, n, s);
  }
  return launched(rc);
}

}  // namespace

extern "C" {

int dyra_dense_create(dyra_dense_t* out, int d_in, int d_out, dyra_dtype_t dtype) {
  if (out == nullptr) return DYRA_ERR_INVALID_ARG;
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_ERR_INVALID_ARG;
  if (d_in < 1 || d_out < 1 || d_in > kMaxRows || d_out > kMaxRows) return DYRA_ERR_INVALID_ARG;
  if (dtype == DYRA_BF16 && (d_in % 8 || d_out % 8)) return DYRA_ERR_ALIGNMENT;
  DeviceInfo dev;
  int rc = current_device_info(&dev);
  if (rc) return rc;
  dyra_dense* p = new (std::nothrow) dyra_dense();
  if (!p) return DYRA_ERR_ALLOC;
  p->d_in = d_in;
  p->d_out = d_out;
  p->dtype = dtype;
  p->dev = dev;
  p->simt = dtype == DYRA_F32 || simt_requested();
  p->n_tiles = p->simt ? 0 : linear_counters(dev);
  Layout l;
  const size_t status = l.add(sizeof(int)), counters = l.add(sizeof(int) * col_sum_blocks(d_out)),
               tiles = l.add(sizeof(int) * p->n_tiles), zeroed = l.total,
               colsum = l.add(sizeof(float) * kColSumChunks * d_out),
               ws = l.add(p->simt ? 0 : linear_ws_bytes(dev));
  if ((rc = allocate(&p->base, l, zeroed))) {
    delete p;
    return rc;
  }
  p->bytes = l.total;
  p->status = part_at<int>(p->base, status);
  p->counters = part_at<int>(p->base, counters);
  p->tiles = part_at<int>(p->base, tiles);
  p->colsum = part_at<float>(p->base, colsum);
  p->ws = part_at<float>(p->base, ws);
  *out = p;
  return DYRA_OK;
}

int dyra_dense_forward(dyra_dense_t p, const void* X, const void* W, const void* bias,
                       const void* residual, int act, void* Y, void* Z, int64_t N,
                       dyra_stream_t stream) {
  if (p == nullptr || N < 0 || N > kMaxRows || !known_act(act)) return DYRA_ERR_INVALID_ARG;
  if (N == 0) return DYRA_OK;
  if (X == nullptr || W == nullptr || Y == nullptr) return DYRA_ERR_INVALID_ARG;
  for (const void* q : {X, W, bias, residual, static_cast<const void*>(Y),
                        static_cast<const void*>(Z)})
    if (!aligned16(q)) return DYRA_ERR_ALIGNMENT;
  const size_t es = elem_size(p->dtype), out = es * N * p->d_out;
  const Span x(X, es * N * p->d_in), w(W, es * p->d_out * p->d_in), b(bias, es * p->d_out),
      r(residual, out), y(Y, out), z(Z, out);
  if (meets_any(y, {x, w, b, z}) || !y.same_or_apart(r) || meets_any(z, {x, w, b, r}))
    return DYRA_ERR_INVALID_ARG;
  DeviceGuard dg(p->dev.device);
  if (!dg.ok) return DYRA_ERR_CUDA;
  LinearGemm g;
  g.A = W;
  g.B = X;
  g.M = p->d_out;
  g.J = N;
  g.K = p->d_in;
  g.bias = bias;
  g.residual = residual;
  g.act = act;
  g.Out = Y;
  g.Z = Z;
  g.status = p->status;
  g.ws = p->ws;
  g.counters = p->tiles;
  g.wait_ns = p->wait_ns;
  return launched(linear(p, g, reinterpret_cast<cudaStream_t>(stream)));
}

int dyra_dense_backward(dyra_dense_t p, const void* dY, const void* X, const void* W,
                        const void* Z, int act, void* dZ, void* dX, void* dW, void* dbias,
                        int64_t N, dyra_stream_t stream) {
  if (p == nullptr || N < 0 || N > kMaxRows || !known_act(act)) return DYRA_ERR_INVALID_ARG;
  const bool has_act = act != DYRA_ACT_NONE;
  if (N > 0 && (dY == nullptr || (dW != nullptr && X == nullptr) ||
                (dX != nullptr && W == nullptr) || (has_act && (Z == nullptr || dZ == nullptr))))
    return DYRA_ERR_INVALID_ARG;
  for (const void* q : {dY, X, W, Z, static_cast<const void*>(dZ), static_cast<const void*>(dX),
                        static_cast<const void*>(dW), static_cast<const void*>(dbias)})
    if (!aligned16(q)) return DYRA_ERR_ALIGNMENT;
  const size_t es = elem_size(p->dtype), out = es * N * p->d_out;
  // what the call reads, and what it writes
  const Span gy(dY, out), x(dW ? X : nullptr, es * N * p->d_in),
      w(dX ? W : nullptr, es * p->d_out * p->d_in), z(has_act ? Z : nullptr, out),
      gz(has_act ? dZ : nullptr, out), gx(dX, es * N * p->d_in), gw(dW, es * p->d_out * p->d_in),
      gb(dbias, es * p->d_out);
  if (!gz.same_or_apart(gy) || !gz.same_or_apart(z) || meets_any(gz, {x, w, gx, gw, gb}) ||
      meets_any(gx, {gy, x, w, z, gw, gb}) || meets_any(gw, {gy, x, w, z, gb}) ||
      meets_any(gb, {gy, x, w, z}))
    return DYRA_ERR_INVALID_ARG;
  DeviceGuard dg(p->dev.device);
  if (!dg.ok) return DYRA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) {
    if ((dW && cudaMemsetAsync(dW, 0, es * p->d_out * p->d_in, s) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, es * p->d_out, s) != cudaSuccess))
      return launched(-1);
    return DYRA_OK;
  }
  if (has_act || dbias) {
    const int rc = p->dtype == DYRA_F32
                       ? act_backward<float>(p, dY, Z, act, dZ, dbias, N, s)
                       : act_backward<__nv_bfloat16>(p, dY, Z, act, dZ, dbias, N, s);
    if (rc) return launched(rc);
  }
  LinearGemm g;
  g.status = p->status;
  g.ws = p->ws;
  g.counters = p->tiles;
  g.wait_ns = p->wait_ns;
  g.B = has_act ? dZ : dY;
  g.M = p->d_in;
  if (dX) {
    g.A = W;
    g.a_mn = true;
    g.J = N;
    g.K = p->d_out;
    g.Out = dX;
    const int rc = linear(p, g, s);
    if (rc) return launched(rc);
  }
  if (dW) {
    g.A = X;
    g.a_mn = g.b_mn = true;
    g.J = p->d_out;
    g.K = N;
    g.Out = dW;
    const int rc = linear(p, g, s);
    if (rc) return launched(rc);
  }
  return DYRA_OK;
}

int dyra_dense_status(dyra_dense_t p) {
  return p == nullptr ? DYRA_ERR_INVALID_ARG : read_status(p->dev, p->status, p->tiles, p->n_tiles);
}

size_t dyra_dense_device_bytes(dyra_dense_t p) { return p == nullptr ? 0 : p->bytes; }

int dyra_dense_destroy(dyra_dense_t p) {
  if (p == nullptr) return DYRA_OK;
  DeviceGuard g(p->dev.device);
  cudaDeviceSynchronize();
  dev_free(p->base);
  delete p;
  return DYRA_OK;
}

int dyra_debug_dense_set_wait_limit(dyra_dense_t p, uint64_t ns) {
  if (p == nullptr) return DYRA_ERR_INVALID_ARG;
  if (p->simt) return DYRA_ERR_UNSUPPORTED;
  p->wait_ns = ns;
  return DYRA_OK;
}

int dyra_moe_create(dyra_moe_t* out, int d_model, int d_ff, int experts, int top_k, int act,
                    int renorm, dyra_dtype_t dtype) {
  if (out == nullptr) return DYRA_ERR_INVALID_ARG;
  if (dtype != DYRA_F32 && dtype != DYRA_BF16) return DYRA_ERR_INVALID_ARG;
  if (d_model < 1 || d_ff < 1 || d_model > DYRA_MOE_MAX_WIDTH || d_ff > DYRA_MOE_MAX_WIDTH ||
      experts < 1 ||
      experts > DYRA_MOE_MAX_EXPERTS || top_k < 1 || top_k > DYRA_MOE_MAX_TOP_K ||
      top_k > experts || !known_act(act) || (renorm != 0 && renorm != 1))
    return DYRA_ERR_INVALID_ARG;
  if (dtype == DYRA_BF16 && (d_model % 8 || d_ff % 8)) return DYRA_ERR_ALIGNMENT;
  DeviceInfo dev;
  int rc = current_device_info(&dev);
  if (rc) return rc;
  dyra_moe* p = new (std::nothrow) dyra_moe();
  if (!p) return DYRA_ERR_ALLOC;
  p->m = MoeShape{d_model, d_ff, experts, top_k, act, renorm};
  p->dtype = dtype;
  p->dev = dev;
  p->simt = dtype == DYRA_F32 || simt_requested();
  const size_t slots = static_cast<size_t>(kMoeTokens) * top_k;
  const size_t hidden_rows =
      p->simt ? slots : static_cast<size_t>(kMoeTokens) * moe_reached_max(p->m);
  const size_t part_bytes = p->simt ? slots * d_model * sizeof(float) : moe_ws_bytes(p->m, dev);
  p->n_tiles = moe_route_counters() + (p->simt ? 0 : moe_counters(p->m));
  Layout l;
  const size_t status = l.add(sizeof(int)), tiles = l.add(sizeof(int) * p->n_tiles),
               zeroed = l.total, hidden = l.add(hidden_rows * d_ff * elem_size(dtype)),
               part = l.add(part_bytes), logits = l.add(moe_logit_bytes(p->m));
  if ((rc = allocate(&p->base, l, zeroed))) {
    delete p;
    return rc;
  }
  p->bytes = l.total;
  p->status = part_at<int>(p->base, status);
  p->tiles = part_at<int>(p->base, tiles);
  p->hidden = part_at<char>(p->base, hidden);
  p->part = part_at<float>(p->base, part);
  p->logits = part_at<double>(p->base, logits);
  *out = p;
  return DYRA_OK;
}

int dyra_moe_route(dyra_moe_t p, const void* X, const void* Wr, int32_t* ids, float* weights,
                   int64_t N, dyra_stream_t stream) {
  const int rc = moe_check(p, N);
  if (rc || N == 0) return rc;
  if (X == nullptr || Wr == nullptr || ids == nullptr || weights == nullptr)
    return DYRA_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Wr) || !aligned16(ids) || !aligned16(weights))
    return DYRA_ERR_ALIGNMENT;
  const Span i = slots_of(p, ids, N), w = slots_of(p, weights, N);
  if (meets_any(i, {rows_of(p, X, N), router_of(p, Wr), w}) ||
      meets_any(w, {rows_of(p, X, N), router_of(p, Wr)}))
    return DYRA_ERR_INVALID_ARG;
  DeviceGuard g(p->dev.device);
  if (!g.ok) return DYRA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(p->dtype == DYRA_F32
                      ? moe_route<float>(p, X, Wr, ids, weights, N, s)
                      : moe_route<__nv_bfloat16>(p, X, Wr, ids, weights, N, s));
}

int dyra_moe_experts(dyra_moe_t p, const void* X, const int32_t* ids, const float* weights,
                     const void* Wgu, const void* Wd, const void* residual, void* Y, int64_t N,
                     dyra_stream_t stream) {
  return run_experts(p, X, ids, weights, Wgu, Wd, residual, Y, N,
                     reinterpret_cast<cudaStream_t>(stream));
}

int dyra_moe_forward(dyra_moe_t p, const void* X, const void* Wr, const void* Wgu, const void* Wd,
                     const void* residual, void* Y, int32_t* ids, float* weights, int64_t N,
                     dyra_stream_t stream) {
  int rc = moe_check(p, N);
  if (rc || N == 0) return rc;
  // the experts' arguments are refused before the router is enqueued
  if (Wgu == nullptr || Wd == nullptr || Y == nullptr) return DYRA_ERR_INVALID_ARG;
  if (!aligned16(Wgu) || !aligned16(Wd) || !aligned16(residual) || !aligned16(Y))
    return DYRA_ERR_ALIGNMENT;
  const Span y = rows_of(p, Y, N), r = rows_of(p, residual, N), i = slots_of(p, ids, N),
             w = slots_of(p, weights, N), gu = experts_of(p, Wgu, 2), dn = experts_of(p, Wd, 1);
  if (meets_any(y, {rows_of(p, X, N), router_of(p, Wr), i, w, gu, dn}) || !y.same_or_apart(r) ||
      meets_any(i, {gu, dn, r}) || meets_any(w, {gu, dn, r}))
    return DYRA_ERR_INVALID_ARG;
  rc = dyra_moe_route(p, X, Wr, ids, weights, N, stream);
  if (rc) return rc;
  return run_experts(p, X, ids, weights, Wgu, Wd, residual, Y, N,
                     reinterpret_cast<cudaStream_t>(stream));
}

int dyra_moe_status(dyra_moe_t p) {
  return p == nullptr ? DYRA_ERR_INVALID_ARG : read_status(p->dev, p->status, p->tiles, p->n_tiles);
}

size_t dyra_moe_device_bytes(dyra_moe_t p) { return p == nullptr ? 0 : p->bytes; }

int dyra_moe_destroy(dyra_moe_t p) {
  if (p == nullptr) return DYRA_OK;
  DeviceGuard g(p->dev.device);
  cudaDeviceSynchronize();
  dev_free(p->base);
  delete p;
  return DYRA_OK;
}

int dyra_debug_moe_set_wait_limit(dyra_moe_t p, uint64_t ns) {
  if (p == nullptr) return DYRA_ERR_INVALID_ARG;
  if (p->simt) return DYRA_ERR_UNSUPPORTED;
  p->wait_ns = ns;
  return DYRA_OK;
}

}  // extern "C"
