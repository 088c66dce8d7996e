// Root-mean-square norm with the residual's addition, its MXFP8 output, and its
// backward pass.  Per token row t over d columns:
//   s = round(x + residual)            (storage type; s = x without a residual)
//   inv = 1 / sqrt(mean_j s_j^2 + eps)
//   y_j = round(s_j inv w_j),  q, sf = MXFP8(y)
// The norm is taken of the rounded sum, so y is a function of what is kept (s,
// inv) and the backward pass recomputes the same xhat = s inv.  Sums are fp32.
//
// Backward, for dy = dL/dy and dsum = dL/ds through the residual stream:
//   c = mean_j(w_j dy_j xhat_j),  dx_j = inv (w_j dy_j - xhat_j c) + dsum_j
//   dw_j = sum_t dy_tj xhat_tj
// (dx is the gradient of x and of the residual: both enter by the sum.)
//
// Both passes are bound by memory: a row is read once, kept in registers over
// the reduction, and written once.  8192 x 6144 bf16 with the residual and the
// MXFP8 output: 70 us, 6.5 TB/s, what a copy reaches; 16 x 2048: 1.5 us in a graph.  Backward
// of the same size with dsum: 77 us a pass, 5.5 TB/s in the first of its two launches
// (a CTA per row and a register per value, which left no room for the next row's
// loads: 641 us).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "quant.cuh"

namespace moe {

// Sum of v over the threads of one row (blockDim.x of them, a multiple of 32)
// in a fixed order; red: shared scratch of 32 floats per row of the block.
MOE_DEV float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// One vector of the output: y = s inv w rounded, and (kMx) its share of the
// MXFP8 block.  A 32-column block is four vectors of four neighbouring lanes;
// the codes are those of the rounded y, so a later quantisation of y gives the
// same bytes.  Every lane of the warp calls.
template <typename T, bool kMx>
MOE_DEV void norm_emit(const float* f, float inv, const uint4& wraw, bool active, int v, size_t row,
                       int d, T* y, uint8_t* yq, uint8_t* ysf) {
  constexpr int VN = Vec16<T>::kN;
  float w[VN], o[VN];
  unpack16(wraw, w, T());
#pragma unroll
  for (int i = 0; i < VN; ++i) o[i] = f[i] * inv * w[i];
  const uint4 packed = pack16(o, T());
  if (active && y) reinterpret_cast<uint4*>(y + row * d)[v] = packed;
  if constexpr (kMx) {
    unpack16(packed, o, T());
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < VN; ++i) amax = fmaxf(amax, fabsf(o[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int s = mx_scale_exp(amax);
    const float is = mx_inv_scale(s);
    uint32_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      q[h] = (uint32_t)mx_quant_inv(o[4 * h], is) | ((uint32_t)mx_quant_inv(o[4 * h + 1], is) << 8) |
             ((uint32_t)mx_quant_inv(o[4 * h + 2], is) << 16) |
             ((uint32_t)mx_quant_inv(o[4 * h + 3], is) << 24);
    if (active) {
      reinterpret_cast<uint2*>(yq + row * d)[v] = make_uint2(q[0], q[1]);
      if ((v & 3) == 0) ysf[row * (d / 32) + (v >> 2)] = mx_scale_byte(s);
    }
  }
}

// One row a CTA; VPT vectors of it per thread in registers, or VPT = 0: rows longer
// than the registers hold are read a second time (from the stored sum when there is
// a residual).  Outputs may share memory with inputs of the same row: a thread reads
// its vectors before it writes them.
template <typename T, int VPT, bool kRes, bool kMx>
__global__ void __launch_bounds__(1024)
rmsnorm_kernel(const T* x, const T* res, const T* __restrict__ w, float eps, int d, T* sum_out,
               T* y, float* inv_out, uint8_t* yq, uint8_t* ysf) {
  pdl_trigger();
  pdl_wait();
  constexpr int VN = Vec16<T>::kN;
  __shared__ float red[32];
  const size_t row = blockIdx.x;
  const int nvec = d / VN, tid = threadIdx.x, step = blockDim.x;
  const uint4* xv = reinterpret_cast<const uint4*>(x + row * d);
  const uint4* rv = kRes ? reinterpret_cast<const uint4*>(res + row * d) : nullptr;
  uint4* sv = kRes ? reinterpret_cast<uint4*>(sum_out + row * d) : nullptr;
  const uint4* wv = reinterpret_cast<const uint4*>(w);
  float ss = 0.f;
  // s of one vector: the rounded sum, stored when there is a residual
  auto take = [&](const uint4& a, const uint4& b, int v, float* f) -> uint4 {
    unpack16(a, f, T());
    uint4 packed = a;
    if constexpr (kRes) {
      float g[VN];
      unpack16(b, g, T());
#pragma unroll
      for (int i = 0; i < VN; ++i) f[i] += g[i];
      packed = pack16(f, T());
      unpack16(packed, f, T());
      sv[v] = packed;
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) ss = fmaf(f[i], f[i], ss);
    return packed;
  };
  if constexpr (VPT > 0) {
    uint4 a[VPT], b[VPT], wr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      a[i] = make_uint4(0, 0, 0, 0);
      b[i] = wr[i] = a[i];
      if (v < nvec) {
        a[i] = xv[v];
        if constexpr (kRes) b[i] = rv[v];
        wr[i] = __ldg(wv + v);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      float f[VN];
      if (v < nvec) a[i] = take(a[i], b[i], v, f);
    }
    ss = row_sum(ss, red);
    const float inv = 1.0f / sqrtf(ss / (float)d + eps);
    if (tid == 0 && inv_out) inv_out[row] = inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      float f[VN];
      unpack16(a[i], f, T());
      norm_emit<T, kMx>(f, inv, wr[i], v < nvec, v, row, d, y, yq, ysf);
    }
  } else {
    for (int v = tid; v < nvec; v += step) {
      float f[VN];
      const uint4 zero = make_uint4(0, 0, 0, 0);
      take(xv[v], kRes ? rv[v] : zero, v, f);
    }
    ss = row_sum(ss, red);
    const float inv = 1.0f / sqrtf(ss / (float)d + eps);
    if (tid == 0 && inv_out) inv_out[row] = inv;
    const uint4* again = kRes ? sv : xv;
    for (int v0 = 0; v0 < nvec; v0 += step) {
      const int v = v0 + tid;
      const bool active = v < nvec;
      uint4 a = make_uint4(0, 0, 0, 0), wr = a;
      if (active) {
        a = again[v];
        wr = __ldg(wv + v);
      }
      float f[VN];
      unpack16(a, f, T());
      norm_emit<T, kMx>(f, inv, wr, active, v, row, d, y, yq, ysf);
    }
  }
}

// Backward: the CTA's blockDim.y row groups take rows base + group, base advancing
// by the grid; a thread owns the same columns in every row, so dw accumulates in
// registers and a CTA writes one fp32 partial row.  A thread copies its own
// vectors of s, dy and dsum into its own slots of a shared-memory ring kDepth - 1
// rows ahead (cp.async, no barrier: nobody else reads them), so the copies of the
// next rows run under this row's reduction, which is the only block-wide wait.
// VPT = 0: rows longer than the ring holds; they are read twice and the partial
// row is kept in global memory (each thread adds to its own columns).
// Rows in the ring: four vectors a thread (wide rows) leave room for two.
__host__ __device__ constexpr int bwd_depth(int vpt) { return vpt == 4 ? 2 : 3; }

// Threads of a CTA at most: up to two vectors a thread, two CTAs of an SM share its registers.
constexpr int bwd_threads(int vpt) { return vpt == 1 || vpt == 2 ? 384 : 512; }

template <typename T, int VPT, bool kSum>
__global__ void __launch_bounds__(bwd_threads(VPT), VPT == 1 || VPT == 2 ? 2 : 1)
rmsnorm_bwd_kernel(const T* s, const T* __restrict__ w, const float* __restrict__ inv_rms,
                   const T* dy, const T* dsum, int rows, int d, T* dx, float* __restrict__ part) {
  pdl_trigger();
  pdl_wait();
  constexpr int VN = Vec16<T>::kN;
  __shared__ float red[2][32 * 8];
  const int nvec = d / VN, tid = threadIdx.x, step = blockDim.x;
  const uint4* wv = reinterpret_cast<const uint4*>(w);
  float* mine = part + (size_t)blockIdx.x * d;
  int flip = 0;
  if constexpr (VPT > 0) {
    constexpr int kIn = kSum ? 3 : 2, kDepth = bwd_depth(VPT);
    extern __shared__ uint4 ring[];  // [kDepth][kIn][VPT][threads]
    const int threads = blockDim.x * blockDim.y, me = threadIdx.y * blockDim.x + tid;
    // unsigned: the fetch runs past a row count next to 2^31
    const unsigned n_rows = rows, stride = gridDim.x * blockDim.y;
    const unsigned first = blockIdx.x * blockDim.y + threadIdx.y;
    auto slot = [&](int stage, int in, int i) -> uint4* {
      return ring + (size_t)((stage * kIn + in) * VPT + i) * threads + me;
    };
    auto fetch = [&](unsigned r, int stage) {
      if (r < n_rows) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = tid + i * step;
          if (v < nvec) {
            const size_t at = (size_t)r * d + (size_t)v * VN;
            cp_async16(slot(stage, 0, i), s + at);
            cp_async16(slot(stage, 1, i), dy + at);
            if constexpr (kSum) cp_async16(slot(stage, 2, i), dsum + at);
          }
        }
      }
      cp_async_commit();
    };
    constexpr int VP = VN / 2;  // pairs of a vector
    uint4 wr[VPT];
    uint64_t dw[VPT][VP];
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) fetch(first + k * stride, k);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      wr[i] = v < nvec ? __ldg(wv + v) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < VP; ++k) dw[i][k] = 0;
    }
    int stage = 0;
    // the loop runs by the CTA's first row: its groups keep step with one another
    for (unsigned base = blockIdx.x * blockDim.y, r = first; base < n_rows;
         base += stride, r += stride) {
      const int ahead = stage ? stage - 1 : kDepth - 1;  // the slots of the row before
      fetch(r + (kDepth - 1) * stride, ahead);
      const bool live = r < n_rows;
      const float inv = live ? inv_rms[r] : 0.f;
      cp_async_wait<kDepth - 1>();
      const uint64_t inv2 = f2_pack(inv, inv);
      uint64_t xh[VPT][VP], wg[VPT][VP], c2 = 0;  // xhat and w dy, kept over the reduction
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * step;
        if (live && v < nvec) {
          uint64_t g[VP];
          unpack16_f2(*slot(stage, 0, i), xh[i], T());
          unpack16_f2(*slot(stage, 1, i), g, T());
          unpack16_f2(wr[i], wg[i], T());
#pragma unroll
          for (int k = 0; k < VP; ++k) {
            xh[i][k] = f2_mul(xh[i][k], inv2);
            wg[i][k] = f2_mul(wg[i][k], g[k]);
            c2 = f2_fma(wg[i][k], xh[i][k], c2);
            dw[i][k] = f2_fma(g[k], xh[i][k], dw[i][k]);
          }
        }
      }
      float c, c_odd;
      f2_unpack(c2, c, c_odd);
      c = row_sum(c + c_odd, red[flip] + 32 * threadIdx.y) / (float)d;
      flip ^= 1;
      const uint64_t minus_c = f2_pack(-c, -c);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * step;
        if (!live || v >= nvec) continue;
        uint64_t o[VP];
        if constexpr (kSum) unpack16_f2(*slot(stage, 2, i), o, T());
#pragma unroll
        for (int k = 0; k < VP; ++k) {
          const uint64_t t = f2_fma(xh[i][k], minus_c, wg[i][k]);
          o[k] = kSum ? f2_fma(t, inv2, o[k]) : f2_mul(t, inv2);
        }
        reinterpret_cast<uint4*>(dx + (size_t)r * d)[v] = pack16_f2<T>(o);
      }
      stage = stage + 1 == kDepth ? 0 : stage + 1;
    }
    // one partial row a CTA: the groups' sums joined in group order
    if (blockDim.y > 1) {
      cp_async_wait<0>();
      __syncthreads();
      uint64_t* all = reinterpret_cast<uint64_t*>(ring);  // [group][VPT][VP][blockDim.x]
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < VP; ++k)
          all[((threadIdx.y * VPT + i) * VP + k) * step + tid] = dw[i][k];
      __syncthreads();
      if (threadIdx.y > 0) return;
      const uint64_t one = f2_pack(1.f, 1.f);
      for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int k = 0; k < VP; ++k)
            dw[i][k] = f2_fma(all[((y * VPT + i) * VP + k) * step + tid], one, dw[i][k]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * step;
      if (v >= nvec) continue;
#pragma unroll
      for (int k = 0; k < VP; k += 2)
        reinterpret_cast<ulonglong2*>(mine)[(v * VN) / 4 + k / 2] =
            make_ulonglong2(dw[i][k], dw[i][k + 1]);
    }
  } else {
    for (int j = tid; j < nvec; j += step)
#pragma unroll
      for (int k = 0; k < VN; ++k) mine[j * VN + k] = 0.f;
    for (int r = blockIdx.x; r < rows; r += gridDim.x) {
      const uint4* srow = reinterpret_cast<const uint4*>(s + (size_t)r * d);
      const uint4* yrow = reinterpret_cast<const uint4*>(dy + (size_t)r * d);
      const float inv = inv_rms[r];
      float c = 0.f;
      for (int v = tid; v < nvec; v += step) {
        float f[VN], g[VN], ww[VN];
        unpack16(srow[v], f, T());
        unpack16(yrow[v], g, T());
        unpack16(__ldg(wv + v), ww, T());
#pragma unroll
        for (int k = 0; k < VN; ++k) {
          const float p = g[k] * (f[k] * inv);
          c = fmaf(ww[k], p, c);
          mine[v * VN + k] += p;
        }
      }
      c = row_sum(c, red[flip]) / (float)d;
      flip ^= 1;
      for (int v = tid; v < nvec; v += step) {
        float f[VN], g[VN], ww[VN], o[VN];
        unpack16(srow[v], f, T());
        unpack16(yrow[v], g, T());
        unpack16(__ldg(wv + v), ww, T());
        if constexpr (kSum)
          unpack16(reinterpret_cast<const uint4*>(dsum + (size_t)r * d)[v], o, T());
#pragma unroll
        for (int k = 0; k < VN; ++k) {
          const float t = inv * (ww[k] * g[k] - f[k] * inv * c);
          o[k] = kSum ? o[k] + t : t;
        }
        reinterpret_cast<uint4*>(dx + (size_t)r * d)[v] = pack16(o, T());
      }
    }
  }
}

// dw[j] = sum over the n partial rows in a fixed order: 32 columns a CTA, 32
// warps that each sum every 32nd row, joined by one warp a column.  An fp32 dw is summed
// in fp64: its error against 64 bits is 5.2e-8 of its norm at 333 x 1000 and 6.7e-8 at
// 4096 x 2048 (7.0e-8 and 1.0e-7 with the warps' sums in fp32), the time 5.78 against 5.75 us.
// A bf16 one gains nothing by it and stays in fp32.  n = 0 gives 0.
template <typename T>
__global__ void __launch_bounds__(1024)
rmsnorm_dw_kernel(const float* __restrict__ part, int n, int d, T* __restrict__ dw) {
  pdl_trigger();
  pdl_wait();
  using Sum = std::conditional_t<sizeof(T) == 4, double, float>;
  __shared__ Sum acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane, mine = blockIdx.x * 32 + warp;
  Sum v = 0;
  if (j < d) {
#pragma unroll 8
    for (int r = warp; r < n; r += 32) v += part[(size_t)r * d + j];
  }
  acc[warp][lane] = v;
  __syncthreads();
  Sum t = acc[lane][warp];
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0 && mine < d) dw[mine] = Cvt<T>::from_f((float)t);
}

}  // namespace moe
