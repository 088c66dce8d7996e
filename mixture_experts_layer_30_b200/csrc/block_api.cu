// C ABI of the operators around the layer (declared in moe.h): the residual RMS
// norm and its backward pass, the 4-bit expert products, and the global gradient
// norm with clipping -- argument validation, workspace layout and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <nvtx3/nvToolsExt.h>

#include "api_shared.h"
#include "clip.cuh"
#include "common.cuh"
#include "moe.h"
#include "norm.cuh"
#include "w4.cuh"

namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

moe_status fail(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(moe::api::error_buffer(), moe::api::kErrorBytes, fmt, ap);
  va_end(ap);
  return st;
}

moe_status launched(cudaError_t launch, const char* what) {
  moe::note_launch();
  const cudaError_t e = cudaGetLastError();
  if (launch == cudaSuccess) launch = e;
  if (launch != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(launch));
  return MOE_OK;
}

#define MOE_TRY(expr)                 \
  do {                                \
    moe_status _s = (expr);           \
    if (_s != MOE_OK) return _s;      \
  } while (0)

#define MOE_ENTRY(name)               \
  moe::api::error_buffer()[0] = 0;    \
  Range nvtx_range_(name)

moe_status need(const void* p, const char* name, size_t align) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail(MOE_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, align);
  return MOE_OK;
}
moe_status optional(const void* p, const char* name, size_t align) {
  return p ? need(p, name, align) : MOE_OK;
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kMaxDevices = 64;
int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : -1;
}

// SMs of the current device, asked for once per device.
int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = current_device();
  int n = dev >= 0 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (dev < 0 ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Lets a kernel take up to `most` bytes of dynamic shared memory: set once per device (one
// value for every call, so that calls of several threads cannot undo one another's).
template <auto* kKernel>
cudaError_t allow_smem(int most) {
  static std::atomic<bool> done[kMaxDevices];
  const int dev = current_device();
  if (dev >= 0 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess && dev >= 0) done[dev].store(true, std::memory_order_release);
  return e;
}

moe_status need_ws(void* ws, size_t have, size_t want) {
  MOE_TRY(need(ws, "workspace", 256));
  if (have < want)
    return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, want);
  return MOE_OK;
}

// --- RMS norm -----------------------------------------------------------------

moe_status check_rows(int32_t T, int32_t d, int32_t dtype) {
  if (dtype != MOE_F32 && dtype != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "dtype %d is neither MOE_F32 nor MOE_BF16", dtype);
  if (T < 0 || d < 1) return fail(MOE_ERR_INVALID_ARG, "bad shape T=%d d=%d", T, d);
  const int vec = dtype == MOE_BF16 ? 8 : 4;
  if (d % vec)
    return fail(MOE_ERR_UNSUPPORTED, "d=%d must be a multiple of %d for 16-byte rows", d, vec);
  return MOE_OK;
}

struct NormArgs {
  const void *x, *res, *w;
  float eps;
  int T, d;
  void *sum, *y;
  float* inv;
  uint8_t *yq, *ysf;
  cudaStream_t st;
};

template <typename T, int VPT, bool kRes, bool kMx>
cudaError_t norm_launch(const NormArgs& a, int threads) {
  return moe::launch_pdl(moe::rmsnorm_kernel<T, VPT, kRes, kMx>, dim3(a.T), dim3(threads), 0, a.st,
                         static_cast<const T*>(a.x), static_cast<const T*>(a.res),
                         static_cast<const T*>(a.w), a.eps, a.d, static_cast<T*>(a.sum),
                         static_cast<T*>(a.y), a.inv, a.yq, a.ysf);
}

template <typename T, bool kRes, bool kMx>
cudaError_t norm_dispatch(const NormArgs& a) {
  const int nvec = a.d / moe::Vec16<T>::kN;
  // threads of one row for vpt vectors each, a whole number of warps
  auto width = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
  if (width(1) <= 256) return norm_launch<T, 1, kRes, kMx>(a, width(1));
  if (width(2) <= 256) return norm_launch<T, 2, kRes, kMx>(a, width(2));
  if (width(4) <= 1024) return norm_launch<T, 4, kRes, kMx>(a, width(4));
  return norm_launch<T, 0, kRes, kMx>(a, 1024);
}

template <typename T>
cudaError_t norm_typed(const NormArgs& a) {
  if constexpr (sizeof(T) == 2) {
    if (a.yq)
      return a.res ? norm_dispatch<T, true, true>(a) : norm_dispatch<T, false, true>(a);
  }
  return a.res ? norm_dispatch<T, true, false>(a) : norm_dispatch<T, false, false>(a);
}

// Rows of partial weight gradients the backward pass writes at most; also its
// largest grid.
constexpr int kNormBwdCtas = 148 * 4;
int norm_bwd_ctas(int T) { return std::min(T, kNormBwdCtas); }

struct NormBwdArgs {
  const void *s, *w, *dy, *dsum;
  const float* inv;
  int T, d;
  void* dx;
  float* part;
  cudaStream_t st;
};

// threads of one row x groups; VPT = 0 takes no ring.  *ctas: partial rows written.
template <typename T, int VPT, bool kSum>
cudaError_t norm_bwd_launch(const NormBwdArgs& a, int threads, int groups, int* ctas) {
  auto* kernel = moe::rmsnorm_bwd_kernel<T, VPT, kSum>;
  const int smem = moe::bwd_depth(VPT) * (kSum ? 3 : 2) * VPT * threads * groups * 16;
  // CTAs an SM: what the ring leaves room for, 1024 threads and four CTAs at most.  Registers
  // may let fewer reside at once; a CTA takes every *ctas-th group of rows either way.
  const int fit = smem ? (224 * 1024) / (smem + 2048) : 4;
  const int per_sm = std::max(1, std::min({4, fit, 1024 / (threads * groups)}));
  *ctas = std::min((a.T + groups - 1) / groups, std::min(sm_count() * per_sm, kNormBwdCtas));
  const cudaError_t e = allow_smem<moe::rmsnorm_bwd_kernel<T, VPT, kSum>>(222 * 1024);
  if (e != cudaSuccess) return e;
  return moe::launch_pdl(kernel, dim3(*ctas), dim3(threads, groups), smem, a.st,
                         static_cast<const T*>(a.s), static_cast<const T*>(a.w), a.inv,
                         static_cast<const T*>(a.dy), static_cast<const T*>(a.dsum), a.T, a.d,
                         static_cast<T*>(a.dx), a.part);
}

template <typename T, bool kSum>
cudaError_t norm_bwd_dispatch(const NormBwdArgs& a, int* ctas) {
  const int nvec = a.d / moe::Vec16<T>::kN;
  auto width = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
  // short rows: several to a CTA of 256 threads
  auto groups = [&](int threads) { return std::max(1, std::min(8, 256 / threads)); };
  if (width(1) <= 128) return norm_bwd_launch<T, 1, kSum>(a, width(1), groups(width(1)), ctas);
  if (width(2) <= 384) return norm_bwd_launch<T, 2, kSum>(a, width(2), groups(width(2)), ctas);
  if (width(4) <= 512) return norm_bwd_launch<T, 4, kSum>(a, width(4), 1, ctas);
  return norm_bwd_launch<T, 0, kSum>(a, 512, 1, ctas);
}

template <typename T>
moe_status norm_bwd_typed(const NormBwdArgs& a, void* dweight) {
  int ctas = 0;
  if (a.T > 0)
    MOE_TRY(launched(a.dsum ? norm_bwd_dispatch<T, true>(a, &ctas)
                            : norm_bwd_dispatch<T, false>(a, &ctas),
                     "RMS norm backward"));
  return launched(moe::launch_pdl(moe::rmsnorm_dw_kernel<T>, dim3((a.d + 31) / 32), dim3(1024), 0,
                                  a.st, a.part, ctas, a.d, static_cast<T*>(dweight)),
                  "RMS norm weight gradient");
}

size_t norm_ws_bytes(int T, int d) {
  return 256 + align256((size_t)std::max(1, norm_bwd_ctas(T)) * d * sizeof(float));
}

// --- 4-bit experts ----------------------------------------------------------------

moe_status check_group(int32_t group) {
  if (group != 32 && group != 64 && group != 128)
    return fail(MOE_ERR_UNSUPPORTED, "group %d is none of 32, 64, 128", group);
  return MOE_OK;
}

struct W4Args {
  const void* a;
  const int32_t* a_rows;
  const void *q0, *s0, *q1, *s1;
  const int32_t* offsets;
  int rows;  // routed rows that the buffers hold
  int n_out, k_dim, gps;
  void* c;
  uint32_t* status;
  cudaStream_t st;
};

template <typename T, bool kGated>
moe_status w4_simt(const moe_shape& s, const W4Args& a) {
  const long long max_rows = (long long)s.T * s.K;
  const long long ncol = (a.n_out + moe::kW4Tile - 1) / moe::kW4Tile;
  const long long chunks = s.N + (max_rows + moe::kW4Tile - 1) / moe::kW4Tile;
  const long long grid = std::min(chunks * ncol, (long long)sm_count() * 8);
  return launched(
      moe::launch_pdl(moe::w4_simt_kernel<T, kGated>, dim3((unsigned)grid), dim3(256), 0, a.st,
                      static_cast<const T*>(a.a), static_cast<const uint32_t*>(a.q0),
                      static_cast<const __nv_bfloat16*>(a.s0), static_cast<const uint32_t*>(a.q1),
                      static_cast<const __nv_bfloat16*>(a.s1), a.offsets, s.N, a.rows,
                      a.n_out, a.k_dim, a.gps, static_cast<T*>(a.c), a.status, a.a_rows, s.T),
      kGated ? "4-bit gate/up" : "4-bit down");
}

template <int GPS, bool kGated, int WR, int MaxNT>
moe_status w4_launch(const moe::W4Problem& p, long long items, cudaStream_t st) {
  auto* kernel = moe::w4_mma_kernel<GPS, kGated, WR, MaxNT>;
  constexpr int fixed = moe::W4Cfg<GPS, WR, MaxNT>::kBytes;
  auto table = [](int n) { return (2 * (n + 1) + 33) * (int)sizeof(int); };
  const int smem = fixed + table(p.N);
  const cudaError_t e = allow_smem<moe::w4_mma_kernel<GPS, kGated, WR, MaxNT>>(
      fixed + table(moe::kMaxExperts));
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "4-bit product: %s", cudaGetErrorString(e));
  const dim3 grid((unsigned)std::min(items, 2LL * sm_count()));
  return launched(moe::launch_pdl(kernel, grid, dim3(moe::kW4Warps * 32), smem, st, p),
                  kGated ? "4-bit gate/up" : "4-bit down");
}

template <int GPS, bool kGated>
moe_status w4_mma(const moe_shape& s, const W4Args& a) {
  const moe::W4Problem p{{static_cast<const uint8_t*>(a.q0), static_cast<const uint8_t*>(a.q1)},
                         {static_cast<const __nv_bfloat16*>(a.s0),
                          static_cast<const __nv_bfloat16*>(a.s1)},
                         static_cast<const __nv_bfloat16*>(a.a), a.a_rows, a.offsets, s.N,
                         a.rows, s.T, a.n_out, a.k_dim, static_cast<__nv_bfloat16*>(a.c),
                         a.status};
  const long long rb = moe::w4_row_blocks(a.n_out), units = kGated ? rb : (rb + 1) / 2;
  const long long max_rows = (long long)s.T * s.K;
  // at most this many row chunks: one per expert that can have rows, one per full chunk
  auto items = [&](int rows, int wr) {
    return (std::min<long long>(s.N, max_rows) + max_rows / rows) * ((units + wr - 1) / wr);
  };
  // Chunks of 8 rows (one column tile) or of 16, by the mean rows of an expert, for gate/up:
  // 3.25 of them (13 tokens at d = 6144, I = 2048, N = 32) 89 against 98 us, 4 (64 tokens of
  // the mid layer) 37 against 31.  Chunks of 32 spread skewed loads worse: 63 against 57 us at
  // 256 tokens of the mid layer.
  if (2 * max_rows <= 7LL * (s.N + s.Z)) {
    // Four pairs in two slices join half as often as two pairs in four, but cut the work in
    // pieces of twice the size: with four pieces and more a CTA (of the experts that K of E
    // choices a token are expected to touch) 46 -> 44 us for the down product of 13 tokens at
    // d = 6144, I = 2048, N = 32; with fewer 87 -> 94 us for its gate/up.
    const double touched = s.N * (1.0 - std::pow(1.0 - (double)s.K / (s.N + s.Z), s.T));
    if (touched * (double)((units + 3) / 4) >= 4.0 * 2 * sm_count())
      return w4_launch<GPS, kGated, 4, 1>(p, items(8, 4), a.st);
    return w4_launch<GPS, kGated, 2, 1>(p, items(8, 2), a.st);
  }
  return w4_launch<GPS, kGated, 4, 2>(p, items(16, 4), a.st);
}

template <bool kGated>
moe_status w4_product(const moe_shape& s, const W4Args& a) {
  if (s.dtype != MOE_BF16) return w4_simt<float, kGated>(s, a);
  switch (a.gps) {
    case 1: return w4_mma<1, kGated>(s, a);
    case 2: return w4_mma<2, kGated>(s, a);
    default: return w4_mma<4, kGated>(s, a);
  }
}

// I is the contraction of the second half: its rows are read 16 bytes at a time.  A chunk's
// end is a 32-bit row number, up to kW4Tile behind the last row, and a block's a 32-bit column.
moe_status check_w4_shape(const moe_shape& s) {
  const int vec = s.dtype == MOE_BF16 ? 8 : 4;
  if (s.I % vec)
    return fail(MOE_ERR_UNSUPPORTED, "I=%d must be a multiple of %d for 16-byte rows", s.I, vec);
  if ((long long)s.T * s.K > 0x7fffffffLL - moe::kW4Tile)
    return fail(MOE_ERR_UNSUPPORTED, "T*K=%lld routed rows leave a chunk's end past int32",
                (long long)s.T * s.K);
  if (std::max(s.d, s.I) > INT32_MAX - moe::kW4Cols)
    return fail(MOE_ERR_UNSUPPORTED, "d=%d, I=%d leave a block's end past int32", s.d, s.I);
  return MOE_OK;
}

// --- gradient norm and clipping -----------------------------------------------------

long long clip_chunks(const moe_grad& g) {
  const int vn = g.dtype == MOE_BF16 ? 8 : 4;
  const long long per = (long long)moe::kClipChunkVecs * vn;
  return std::max(1LL, (g.numel + per - 1) / per);
}

moe_status check_grads(int32_t n, const moe_grad* list, bool writes) {
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n_tensors=%d is negative", n);
  if (n > 0 && !list) return fail(MOE_ERR_INVALID_ARG, "the gradient list is NULL");
  for (int i = 0; i < n; ++i) {
    const moe_grad& g = list[i];
    if (g.dtype != MOE_F32 && g.dtype != MOE_BF16)
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: dtype %d is neither MOE_F32 nor MOE_BF16", i,
                  g.dtype);
    if (g.numel < 0 || g.numel > (1LL << 48))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: numel %lld", i, (long long)g.numel);
    if (g.numel == 0) continue;
    const size_t e = g.dtype == MOE_BF16 ? 2 : 4;
    if (!g.grad || reinterpret_cast<uintptr_t>(g.grad) % e)
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: grad is NULL or misaligned", i);
    if (writes && (!g.out || reinterpret_cast<uintptr_t>(g.out) % e))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: out is NULL or misaligned", i);
  }
  return MOE_OK;
}

// Fills one table from list[at..]; returns the position behind it.
int clip_table(int n, const moe_grad* list, int at, moe::ClipTable* tab) {
  tab->n = 0;
  tab->first[0] = 0;
  for (uint32_t& b : tab->bf16) b = 0;
  for (; at < n && tab->n < moe::kClipTensors; ++at) {
    const moe_grad& g = list[at];
    if (g.numel == 0) continue;
    const int i = tab->n++;
    tab->in[i] = g.grad;
    tab->out[i] = g.out;
    tab->numel[i] = g.numel;
    if (g.dtype == MOE_BF16) tab->bf16[i >> 5] |= 1u << (i & 31);
    tab->first[i + 1] = tab->first[i] + clip_chunks(g);
  }
  return at;
}

unsigned clip_grid(const moe::ClipTable& tab) {
  return (unsigned)std::min<long long>(std::max(1LL, tab.first[tab.n]), moe::kClipMaxCtas);
}

size_t clip_ws_bytes(int n) {
  const int launches = std::max(1, (n + moe::kClipTensors - 1) / moe::kClipTensors);
  return 256 + align256((size_t)launches * moe::kClipMaxCtas * sizeof(double));
}

}  // namespace

extern "C" {

moe_status moe_rmsnorm(int32_t T, int32_t d, int32_t dtype, const void* x, const void* residual,
                       const void* weight, float eps, void* sum_out, void* y, float* inv_rms,
                       void* y_q, void* y_sf, void* stream) {
  MOE_ENTRY("moe_rmsnorm");
  MOE_TRY(check_rows(T, d, dtype));
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(MOE_ERR_INVALID_ARG, "eps=%g must be finite and not negative", (double)eps);
  if (y_q && (dtype != MOE_BF16 || d % 32))
    return fail(MOE_ERR_UNSUPPORTED, "the MXFP8 output needs bf16 and d %% 32 == 0 (d=%d)", d);
  MOE_TRY(need(weight, "weight", 16));
  if (T == 0) return MOE_OK;
  if (!y_q != !y_sf) return fail(MOE_ERR_INVALID_ARG, "y_q and y_sf go together");
  if (!y && !y_q) return fail(MOE_ERR_INVALID_ARG, "neither y nor y_q is given");
  MOE_TRY(need(x, "x", 16));
  MOE_TRY(optional(residual, "residual", 16));
  if (residual) MOE_TRY(need(sum_out, "sum_out", 16));
  if (!residual && sum_out)
    return fail(MOE_ERR_INVALID_ARG, "sum_out is given without a residual");
  MOE_TRY(optional(y, "y", 16));
  MOE_TRY(optional(inv_rms, "inv_rms", 4));
  MOE_TRY(optional(y_q, "y_q", 16));
  if (y && y == sum_out) return fail(MOE_ERR_INVALID_ARG, "y and sum_out are the same buffer");
  const NormArgs a{x, residual, weight, eps, T, d, sum_out, y, inv_rms,
                   static_cast<uint8_t*>(y_q), static_cast<uint8_t*>(y_sf),
                   static_cast<cudaStream_t>(stream)};
  return launched(dtype == MOE_BF16 ? norm_typed<__nv_bfloat16>(a) : norm_typed<float>(a),
                  "RMS norm");
}

size_t moe_rmsnorm_workspace_bytes(int32_t T, int32_t d) {
  if (T < 0 || d < 1) return 0;
  return norm_ws_bytes(T, d);
}

moe_status moe_rmsnorm_backward(int32_t T, int32_t d, int32_t dtype, const void* s,
                                const void* weight, const float* inv_rms, const void* dy,
                                const void* dsum, void* dx, void* dweight, void* ws,
                                size_t ws_bytes, void* stream) {
  MOE_ENTRY("moe_rmsnorm_backward");
  MOE_TRY(check_rows(T, d, dtype));
  MOE_TRY(need_ws(ws, ws_bytes, norm_ws_bytes(T, d)));
  MOE_TRY(need(weight, "weight", 16));
  MOE_TRY(need(dweight, "dweight", 16));
  if (T > 0) {
    MOE_TRY(need(s, "s", 16));
    MOE_TRY(need(inv_rms, "inv_rms", 4));
    MOE_TRY(need(dy, "dy", 16));
    MOE_TRY(optional(dsum, "dsum", 16));
    MOE_TRY(need(dx, "dx", 16));
  }
  const NormBwdArgs a{s, weight, dy, dsum, inv_rms, T, d, dx,
                      reinterpret_cast<float*>(static_cast<char*>(ws) + 256),
                      static_cast<cudaStream_t>(stream)};
  return dtype == MOE_BF16 ? norm_bwd_typed<__nv_bfloat16>(a, dweight)
                           : norm_bwd_typed<float>(a, dweight);
}

size_t moe_w4_code_bytes(int32_t n_mats, int32_t rows, int32_t cols) {
  if (n_mats < 0 || rows < 0 || cols < 0) return 0;
  return (size_t)n_mats * moe::w4_row_blocks(rows) * moe::w4_col_blocks(cols) * moe::kW4Block;
}

size_t moe_w4_scale_bytes(int32_t n_mats, int32_t rows, int32_t cols, int32_t group) {
  if (n_mats < 0 || rows < 0 || cols < 0 || (group != 32 && group != 64 && group != 128)) return 0;
  return moe_w4_code_bytes(n_mats, rows, cols) / moe::kW4Block * moe::kW4Rows *
         (moe::kW4Cols / group) * 2;
}

moe_status moe_quantize_weights_w4(int32_t n_mats, int32_t rows, int32_t cols, int32_t group,
                                   int32_t dtype, const void* src, void* dst_q, void* dst_s,
                                   void* stream) {
  MOE_ENTRY("moe_quantize_weights_w4");
  if (dtype != MOE_F32 && dtype != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "dtype %d is neither MOE_F32 nor MOE_BF16", dtype);
  if (n_mats < 0 || rows < 0 || cols < 0)
    return fail(MOE_ERR_INVALID_ARG, "bad shape n_mats=%d rows=%d cols=%d", n_mats, rows, cols);
  MOE_TRY(check_group(group));
  const long long blocks =
      (long long)n_mats * moe::w4_row_blocks(rows) * moe::w4_col_blocks(cols);
  if (blocks == 0) return MOE_OK;
  if (blocks > 0x7fffffffLL) return fail(MOE_ERR_UNSUPPORTED, "too many weight blocks");
  MOE_TRY(need(src, "src", dtype == MOE_BF16 ? 2 : 4));
  MOE_TRY(need(dst_q, "dst_q", 16));
  MOE_TRY(need(dst_s, "dst_s", 16));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto* kernel, auto* p) {
    return moe::launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, st, p, rows, cols,
                           moe::kW4Cols / group, static_cast<uint32_t*>(dst_q),
                           static_cast<__nv_bfloat16*>(dst_s));
  };
  return launched(dtype == MOE_BF16
                      ? go(moe::quantize_weights_w4_kernel<__nv_bfloat16>,
                           static_cast<const __nv_bfloat16*>(src))
                      : go(moe::quantize_weights_w4_kernel<float>, static_cast<const float*>(src)),
                  "4-bit weight quantisation");
}

moe_status moe_expert_gate_up_w4(const moe_shape* shape, int32_t group, const void* x,
                                 const int32_t* row_token, const void* w1_q, const void* w1_s,
                                 const void* w3_q, const void* w3_s, const int32_t* offsets,
                                 void* h, void* ws, size_t ws_bytes, void* stream) {
  const int64_t rows = shape ? (int64_t)shape->T * shape->K : 0;
  // more rows than 32 bits hold: the shape is refused, whatever the count
  return moe_expert_gate_up_w4_rows(shape, group, (int32_t)std::min<int64_t>(rows, INT32_MAX), x,
                                    row_token, w1_q, w1_s, w3_q, w3_s, offsets, h, ws, ws_bytes,
                                    stream);
}

moe_status moe_expert_gate_up_w4_rows(const moe_shape* shape, int32_t group, int32_t n_rows,
                                      const void* x, const int32_t* row_token, const void* w1_q,
                                      const void* w1_s, const void* w3_q, const void* w3_s,
                                      const int32_t* offsets, void* h, void* ws, size_t ws_bytes,
                                      void* stream) {
  MOE_ENTRY("moe_expert_gate_up_w4");
  uint32_t* status = nullptr;
  MOE_TRY(moe::api::layer_status(shape, ws, ws_bytes, &status));
  const moe_shape& s = *shape;
  MOE_TRY(check_group(group));
  MOE_TRY(check_w4_shape(s));
  if (n_rows < 0 || n_rows > (long long)s.T * s.K)
    return fail(MOE_ERR_INVALID_ARG, "n_rows=%d outside [0, T*K=%lld]", n_rows,
                (long long)s.T * s.K);
  MOE_TRY(need(w1_q, "w1_q", 16));
  MOE_TRY(need(w1_s, "w1_s", 16));
  MOE_TRY(need(w3_q, "w3_q", 16));
  MOE_TRY(need(w3_s, "w3_s", 16));
  MOE_TRY(need(offsets, "offsets", 4));
  if (s.T == 0) return MOE_OK;
  MOE_TRY(need(x, "x", 16));
  MOE_TRY(optional(row_token, "row_token", 4));
  MOE_TRY(need(h, "h", 16));
  return w4_product<true>(s, W4Args{x, row_token, w1_q, w1_s, w3_q, w3_s, offsets, n_rows, s.I,
                                    s.d, moe::kW4Cols / group, h, status,
                                    static_cast<cudaStream_t>(stream)});
}

moe_status moe_expert_down_w4(const moe_shape* shape, int32_t group, const void* h,
                              const void* w2_q, const void* w2_s, const int32_t* offsets,
                              void* y_perm, void* ws, size_t ws_bytes, void* stream) {
  MOE_ENTRY("moe_expert_down_w4");
  uint32_t* status = nullptr;
  MOE_TRY(moe::api::layer_status(shape, ws, ws_bytes, &status));
  const moe_shape& s = *shape;
  MOE_TRY(check_group(group));
  MOE_TRY(check_w4_shape(s));
  MOE_TRY(need(w2_q, "w2_q", 16));
  MOE_TRY(need(w2_s, "w2_s", 16));
  MOE_TRY(need(offsets, "offsets", 4));
  if (s.T == 0) return MOE_OK;
  MOE_TRY(need(h, "h", 16));
  MOE_TRY(need(y_perm, "y_perm", 16));
  return w4_product<false>(s, W4Args{h, nullptr, w2_q, w2_s, nullptr, nullptr, offsets, s.T * s.K,
                                     s.d, s.I, moe::kW4Cols / group, y_perm, status,
                                     static_cast<cudaStream_t>(stream)});
}

size_t moe_grad_workspace_bytes(int32_t n_tensors) {
  return n_tensors < 0 ? 0 : clip_ws_bytes(n_tensors);
}

moe_status moe_grad_norm(int32_t n_tensors, const moe_grad* list, float* norm, void* ws,
                         size_t ws_bytes, void* stream) {
  MOE_ENTRY("moe_grad_norm");
  MOE_TRY(check_grads(n_tensors, list, false));
  MOE_TRY(need_ws(ws, ws_bytes, clip_ws_bytes(n_tensors)));
  MOE_TRY(need(norm, "norm", 4));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
  unsigned int* ticket = reinterpret_cast<unsigned int*>(static_cast<char*>(ws) + 4);
  int at = 0, parts = 0;
  do {
    moe::ClipTable tab;
    at = clip_table(n_tensors, list, at, &tab);
    const unsigned grid = clip_grid(tab);
    MOE_TRY(launched(moe::launch_pdl(moe::grad_norm_kernel, dim3(grid), dim3(moe::kClipThreads),
                                     0, st, tab, part, parts, parts + (int)grid, ticket,
                                     at >= n_tensors ? norm : nullptr),
                     "gradient norm"));
    parts += (int)grid;
  } while (at < n_tensors);
  return MOE_OK;
}

moe_status moe_grad_clip(int32_t n_tensors, const moe_grad* list, float max_norm,
                         const float* norm, void* stream) {
  MOE_ENTRY("moe_grad_clip");
  MOE_TRY(check_grads(n_tensors, list, true));
  if (!(max_norm >= 0.f))
    return fail(MOE_ERR_INVALID_ARG, "max_norm=%g must not be negative or NaN", (double)max_norm);
  MOE_TRY(need(norm, "norm", 4));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bool in_place = true;
  for (int i = 0; i < n_tensors; ++i)
    if (list[i].numel > 0 && list[i].grad != list[i].out) in_place = false;
  for (int at = 0; at < n_tensors;) {
    moe::ClipTable tab;
    at = clip_table(n_tensors, list, at, &tab);
    if (tab.n == 0) continue;
    MOE_TRY(launched(moe::launch_pdl(moe::grad_clip_kernel, dim3(clip_grid(tab)),
                                     dim3(moe::kClipThreads), 0, st, tab, max_norm, in_place,
                                     norm),
                     "gradient clipping"));
  }
  return MOE_OK;
}

}  // extern "C"
