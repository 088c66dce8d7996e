// 4-bit expert weights with group scales (W4): the expert products with the
// activations left in their own type.
//   W[n, k] = (code[n, k] - 8) * scale[n, k / G],  code in 0..15, G in {32, 64, 128}
// Scales are bf16: the quantiser divides by the rounded scale, so their rounding
// costs no accuracy beyond that of the 4-bit grid itself.
//
// Layout.  Rows and columns are padded to multiples of 16 and 128 (code 8, scale
// 0: the value 0) and cut into blocks of 16 rows by 128 columns, ordered (matrix,
// row block, column block): 1024 contiguous bytes of codes, 64 a row.  Byte
// 16 t + 4 j .. + 3 of a row is one little-endian word with columns
// 32 j + 8 t .. + 7; nibble p of the word holds column 2 p (p < 4) or 2 (p - 4) + 1
// of those eight.  So the 16 bytes that a lane of a matrix instruction's
// quad t loads hold eight columns of every 32-column piece, and the pair of
// columns 2 i, 2 i + 1 is word >> 4 i under the mask 0x000f000f -- the two halves of
// one packed bf16 operand.  A warp that takes 16 rows streams one contiguous run.
// Scales: [matrix, row block, column block, 16 rows, 128 / G].
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kW4Rows = 16, kW4Cols = 128, kW4Block = 1024;  // one block of codes, bytes

__host__ MOE_DEV int w4_row_blocks(int rows) { return (rows + kW4Rows - 1) / kW4Rows; }
__host__ MOE_DEV int w4_col_blocks(int cols) { return (cols + kW4Cols - 1) / kW4Cols; }

// One CTA per block; a thread takes eight columns of one row.  scale =
// round_bf16(amax / 7), code = 8 + round(w / scale) (nearest even, 0 where the
// scale is 0).
template <typename T>
__global__ void __launch_bounds__(256)
quantize_weights_w4_kernel(const T* __restrict__ src, int rows, int cols, int gps,
                           uint32_t* __restrict__ dst_q, __nv_bfloat16* __restrict__ dst_s) {
  pdl_trigger();
  pdl_wait();
  const int sp_n = w4_col_blocks(cols), rb_n = w4_row_blocks(rows);
  const long long block = blockIdx.x;
  const int sp = (int)(block % sp_n);
  const long long mr = block / sp_n;
  const int rb = (int)(mr % rb_n);
  const long long m = mr / rb_n;
  const int r = threadIdx.x >> 4, c8 = threadIdx.x & 15;
  const int row = rb * kW4Rows + r, col = sp * kW4Cols + c8 * 8;
  float f[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = row < rows && col + i < cols
               ? Cvt<T>::to_f(src[((size_t)m * rows + row) * cols + col + i]) : 0.f;
    amax = fmaxf(amax, fabsf(f[i]));
  }
  const int lanes = 16 / gps;  // threads of one group
  for (int o = 1; o < lanes; o <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const __nv_bfloat16 s16 = __float2bfloat16_rn(amax / 7.0f);
  const float s = __bfloat162float(s16);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = s > 0.f ? fminf(7.f, fmaxf(-8.f, rintf(f[i] / s))) : 0.f;
    w |= (uint32_t)((int)q + 8) << (4 * (i / 2 + 4 * (i & 1)));
  }
  const int j = c8 >> 2, t = c8 & 3;
  dst_q[(size_t)block * (kW4Block / 4) + r * 16 + t * 4 + j] = w;
  if (c8 % lanes == 0)
    dst_s[((size_t)block * kW4Rows + r) * gps + c8 / lanes] = s16;
}

// Expert products on CUDA cores (fp32 layers): the tiling of the row-major
// CUDA-core grouped GEMM, with one 4-bit word decoded per thread and 32 columns.
//   gated: C[r, n] = SiLU(A[r] . B0[e][n]) * (A[r] . B1[e][n]);  plain: A[r] . B0[e][n]
// Row r of A is A[r], or A[a_rows[r]]; fp32 sums.
constexpr int kW4Tile = 64, kW4K = 32;

template <typename T, bool kGated>
__global__ void __launch_bounds__(256)
w4_simt_kernel(const T* __restrict__ A, const uint32_t* __restrict__ q0,
               const __nv_bfloat16* __restrict__ s0, const uint32_t* __restrict__ q1,
               const __nv_bfloat16* __restrict__ s1, const int32_t* __restrict__ offsets, int N,
               int max_rows, int n_out, int k_dim, int gps, T* __restrict__ C, uint32_t* status,
               const int32_t* __restrict__ a_rows, int a_src_rows) {
  pdl_trigger();
  pdl_wait();
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int scan_tmp[33];
  __shared__ float As[kW4K][kW4Tile + 4];
  __shared__ float Bs[kGated ? 2 : 1][kW4K][kW4Tile + 4];
  build_chunk_prefix(offsets, N, max_rows, kW4Tile, prefix, scan_tmp, status);
  const int ncol = (n_out + kW4Tile - 1) / kW4Tile;
  const int rb_n = w4_row_blocks(n_out), sp_n = w4_col_blocks(k_dim);
  const long long total = (long long)prefix[N] * ncol;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int lr = tid >> 2, lt = tid & 3;  // row and eight columns that this thread loads
  for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int chunk = (int)(tile / ncol), col = (int)(tile % ncol);
    const int e = find_expert(prefix, N, chunk);
    const int r0 = offsets[e] + (chunk - prefix[e]) * kW4Tile;
    const int r1 = min(r0 + kW4Tile, (int)offsets[e + 1]);
    const int n0 = col * kW4Tile;
    int src = -1;
    if (r0 + lr < r1) {
      src = a_rows ? a_rows[r0 + lr] : r0 + lr;
      if (a_rows && (src < 0 || src >= a_src_rows)) {
        set_status(status, MOE_DEV_BAD_OFFSETS);
        src = 0;
      }
    }
    const int rb = (n0 + lr) / kW4Rows;
    float acc0[4][4] = {}, acc1[4][4] = {};
    for (int k0 = 0; k0 < k_dim; k0 += kW4K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + lt * 8 + i;
        As[lt * 8 + i][lr] =
            src >= 0 && k < k_dim ? Cvt<T>::to_f(A[(size_t)src * k_dim + k]) : 0.f;
      }
      const size_t block = ((size_t)e * rb_n + rb) * sp_n + k0 / kW4Cols;
      const int r16 = (n0 + lr) % kW4Rows, j = k0 % kW4Cols / 32;
      const int at = r16 * 16 + lt * 4 + j;
      const int sc = r16 * gps + (k0 % kW4Cols + lt * 8) * gps / kW4Cols;
#pragma unroll
      for (int h = 0; h < (kGated ? 2 : 1); ++h) {
        uint32_t w = 0x88888888u;
        float s = 0.f;
        if (rb < rb_n) {
          w = __ldg((h ? q1 : q0) + block * (kW4Block / 4) + at);
          s = __bfloat162float((h ? s1 : s0)[block * kW4Rows * gps + sc]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = (int)(w >> (4 * (i / 2 + 4 * (i & 1))) & 15u) - 8;
          Bs[h][lt * 8 + i][lr] = (float)c * s;
        }
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kW4K; ++kk) {
        float a[4], b[4], g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = As[kk][ty * 4 + i];
          b[i] = Bs[0][kk][tx * 4 + i];
          if (kGated) g[i] = Bs[kGated ? 1 : 0][kk][tx * 4 + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            acc0[i][jj] = fmaf(a[i], b[jj], acc0[i][jj]);
            if (kGated) acc1[i][jj] = fmaf(a[i], g[jj], acc1[i][jj]);
          }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int gr = r0 + ty * 4 + i;
      if (gr >= r1) continue;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int gn = n0 + tx * 4 + jj;
        if (gn >= n_out) continue;
        const float v = kGated ? silu(acc0[i][jj]) * acc1[i][jj] : acc0[i][jj];
        C[(size_t)gr * n_out + gn] = Cvt<T>::from_f(v);
      }
    }
  }
}

}  // namespace moe
