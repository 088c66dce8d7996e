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

// ---------------------------------------------------------------------------
// Expert products on the matrix instructions (bf16 layers)
//
// A decode batch gives an expert a few rows, so the weights are the traffic: an
// expert's codes are streamed once through registers and every other cost has to
// stay below that stream.  The weights are the 16-row operand of
// mma.m16n8k16 (M = output rows), the tokens its 8 columns; up to 4 column tiles
// (32 rows of an expert) share one pass over the codes.
//   * A lane loads 16 bytes of a row: columns 32 j + 8 t .. + 7 for j = 0..3.
//     The order of a contraction is free, so the instruction's k slots are given
//     the columns as they lie: step (j, i) takes 4 of the lane's 8 columns, and
//     the token operand is the matching 16 bytes of the token row.
//   * A code becomes a bf16 exactly: 0x4300 | code is 128 + code, minus 136.
//     Products are exact in fp32; each group's fp32 sum is multiplied by the
//     group's scale in fp32, so the weights are never rounded.
//   * Eight warps take WR pairs of row blocks times 8 / WR slices of the
//     contraction; slices are joined through shared memory in slice order.
//   * Items (row chunk of an expert, WR pairs of row blocks) are cut into equal
//     contiguous runs, one per CTA, and a warp loads the next item's first codes
//     while it still computes this one.
// Token rows are read through L1 (the same 64 bytes by every warp of a slice),
// codes bypass it.
// ---------------------------------------------------------------------------
constexpr int kW4Warps = 8;
constexpr int kW4MaxTokens = 32;  // rows of an expert per pass: 4 column tiles
constexpr int kW4Depth = 2;       // column blocks in flight per warp

MOE_DEV uint4 w4_load_codes(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Columns (2 i, 2 i + 1) of a code word as a packed bf16 pair.
template <int I>
MOE_DEV uint32_t w4_pair(uint32_t w) {
  uint32_t v;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xEA;" : "=r"(v) : "r"(w >> (4 * I)));
  __nv_bfloat162 b = *reinterpret_cast<__nv_bfloat162*>(&v);
  b = __hsub2(b, __nv_bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308)));
  return *reinterpret_cast<uint32_t*>(&b);
}

MOE_DEV void w4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The scales of one row and column block: GPS bf16 values.
template <int GPS> struct W4Scale;
template <> struct W4Scale<1> {
  uint16_t v;
  MOE_DEV void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint16_t*>(p)); }
  MOE_DEV float get(int) const { return __uint_as_float((uint32_t)v << 16); }
};
template <> struct W4Scale<2> {
  uint32_t v;
  MOE_DEV void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint32_t*>(p)); }
  MOE_DEV float get(int i) const {
    return __uint_as_float(i ? v & 0xffff0000u : v << 16);
  }
};
template <> struct W4Scale<4> {
  uint2 v;
  MOE_DEV void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
  MOE_DEV float get(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// One column block of a warp's two row blocks.
template <int GPS>
struct W4Step {
  uint4 q[2][2];            // [row block][rows g / g + 8]
  W4Scale<GPS> s[2][2];
};

struct W4Problem {
  const uint8_t* q[2];           // codes of the two products (plain: one)
  const __nv_bfloat16* s[2];
  const __nv_bfloat16* a;        // token rows
  const int32_t* a_rows;
  const int32_t* offsets;
  int N, max_rows, a_src_rows, n_out, k_dim;
  __nv_bfloat16* c;
  uint32_t* status;
};

struct W4Item {
  long long block[2];  // first block (column block 0) of the two row blocks
  int unit;            // this CTA's first pair of row blocks
  int r0, rows;        // first routed row and how many (<= 32; 0: no item)
  int chunk, group;    // position in the item list
};

template <int NT, int GPS, bool kGated, int WR>
MOE_DEV void w4_item(const W4Problem& p, const W4Item& cur, const W4Item& nxt, int n_steps,
                     W4Step<GPS> (&buf)[kW4Depth], float4* red) {
  constexpr int WK = kW4Warps / WR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3, ks = warp % WK;
  // the token rows of this lane's columns; columns past the last row repeat row 0 of
  // the chunk and are not stored
  const __nv_bfloat16* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = n * 8 + g;
    int row = cur.r0 + (i < cur.rows ? i : 0);
    if (p.a_rows) {
      row = p.a_rows[row];
      if (row < 0 || row >= p.a_src_rows) {
        if (t == 0 && warp == 0) set_status(p.status, MOE_DEV_BAD_OFFSETS);
        row = 0;
      }
    }
    xr[n] = p.a + (size_t)row * p.k_dim + 8 * t;
  }
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[m][n][k] = 0.f;
  const int rounds = (n_steps + kW4Depth - 1) / kW4Depth * kW4Depth;
  for (int i0 = 0; i0 < rounds; i0 += kW4Depth) {
#pragma unroll
    for (int b = 0; b < kW4Depth; ++b) {
      const int i = i0 + b;
      if (i < n_steps) {
        const int k0 = (ks + i * WK) * kW4Cols;
        const W4Step<GPS>& w = buf[b];
        float c[2][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 x[NT];
          const int kj = k0 + 32 * j;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            x[n] = kj + 8 * t < p.k_dim
                       ? __ldg(reinterpret_cast<const uint4*>(xr[n] + kj))
                       : make_uint4(0, 0, 0, 0);
          constexpr int kPer = 4 / GPS;  // 32-column pieces of one group
          if (j % kPer == 0) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) c[m][n][k] = 0.f;
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t lo = j == 0 ? w.q[m][0].x : j == 1 ? w.q[m][0].y
                                : j == 2 ? w.q[m][0].z : w.q[m][0].w;
            const uint32_t hi = j == 0 ? w.q[m][1].x : j == 1 ? w.q[m][1].y
                                : j == 2 ? w.q[m][1].z : w.q[m][1].w;
            {
              const uint32_t a0 = w4_pair<0>(lo), a1 = w4_pair<0>(hi);
              const uint32_t a2 = w4_pair<1>(lo), a3 = w4_pair<1>(hi);
#pragma unroll
              for (int n = 0; n < NT; ++n) w4_mma(c[m][n], a0, a1, a2, a3, x[n].x, x[n].y);
            }
            {
              const uint32_t a0 = w4_pair<2>(lo), a1 = w4_pair<2>(hi);
              const uint32_t a2 = w4_pair<3>(lo), a3 = w4_pair<3>(hi);
#pragma unroll
              for (int n = 0; n < NT; ++n) w4_mma(c[m][n], a0, a1, a2, a3, x[n].z, x[n].w);
            }
            if (j % kPer == kPer - 1) {
              const float s0 = w.s[m][0].get(j / kPer), s1 = w.s[m][1].get(j / kPer);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                acc[m][n][0] = fmaf(s0, c[m][n][0], acc[m][n][0]);
                acc[m][n][1] = fmaf(s0, c[m][n][1], acc[m][n][1]);
                acc[m][n][2] = fmaf(s1, c[m][n][2], acc[m][n][2]);
                acc[m][n][3] = fmaf(s1, c[m][n][3], acc[m][n][3]);
              }
            }
          }
        }
      }
      // refill: a later column block of this item, or one of the next item's first
      const int later = i + kW4Depth;
      const bool same = later < n_steps;
      const int step = same ? later : later - rounds;
      if (same || (step >= 0 && step < n_steps && nxt.rows > 0)) {
        const W4Item& it = same ? cur : nxt;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const long long blk = it.block[m] + ks + step * WK;
          const uint8_t* q = p.q[kGated ? m : 0] + blk * kW4Block + lane * 16;
          const __nv_bfloat16* s = p.s[kGated ? m : 0] + (blk * kW4Rows + g) * GPS;
          buf[b].q[m][0] = w4_load_codes(q);
          buf[b].q[m][1] = w4_load_codes(q + kW4Block / 2);
          buf[b].s[m][0].load(s);
          buf[b].s[m][1].load(s + 8 * GPS);
        }
      }
    }
  }
  // join the slices: slot (warp, row block, column tile) of 32 lanes
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      red[((warp * 2 + m) * NT + n) * 32 + lane] =
          make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
  __syncthreads();
  const int rb_n = w4_row_blocks(p.n_out);
  constexpr int kOut = kGated ? WR * NT : WR * 2 * NT;  // 32-lane pieces of the result
  for (int o = warp; o < kOut; o += kW4Warps) {
    const int n = o % NT, m = kGated ? 0 : o / NT % 2, u = kGated ? o / NT : o / NT / 2;
    auto join = [&](int mm) {
      float4 v = red[((u * WK * 2 + mm) * NT + n) * 32 + lane];
#pragma unroll
      for (int k = 1; k < WK; ++k) {
        const float4 w = red[(((u * WK + k) * 2 + mm) * NT + n) * 32 + lane];
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      return v;
    };
    float4 v = join(m);
    if (kGated) {
      const float4 up = join(1);
      v = make_float4(silu(v.x) * up.x, silu(v.y) * up.y, silu(v.z) * up.z, silu(v.w) * up.w);
    }
    const int rb = kGated ? cur.unit + u : 2 * (cur.unit + u) + m;
    const int i0 = n * 8 + 2 * t, c0 = rb * kW4Rows + g;
    if (rb >= rb_n) continue;
    __nv_bfloat16* out = p.c + (size_t)(cur.r0 + i0) * p.n_out;
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + (k & 1) < cur.rows && c0 + (k >> 1) * 8 < p.n_out)
        out[(size_t)(k & 1) * p.n_out + c0 + (k >> 1) * 8] = __float2bfloat16_rn(f[k]);
  }
}

template <int GPS, bool kGated, int WR>
__global__ void __launch_bounds__(kW4Warps * 32, 2)
w4_mma_kernel(const __grid_constant__ W4Problem p) {
  pdl_trigger();
  pdl_wait();
  constexpr int WK = kW4Warps / WR;
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int scan_tmp[33];
  // two buffers up to two column tiles, one above
  __shared__ float4 red[kW4Warps * 2 * 4 * 32];
  build_chunk_prefix(p.offsets, p.N, p.max_rows, kW4MaxTokens, prefix, scan_tmp, p.status);
  const int rb_n = w4_row_blocks(p.n_out), sp_n = w4_col_blocks(p.k_dim);
  const int units = kGated ? rb_n : (rb_n + 1) / 2;
  const int groups = (units + WR - 1) / WR;
  const long long total = (long long)prefix[p.N] * groups;
  const long long first = total * blockIdx.x / gridDim.x;
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  if (first >= end) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, ks = warp % WK, wu = warp / WK;
  const int n_steps = sp_n > ks ? (sp_n - ks + WK - 1) / WK : 0;
  auto place = [&](int chunk, int group, W4Item* it) {
    it->chunk = chunk;
    it->group = group;
    const int e = find_expert(prefix, p.N, chunk);
    it->r0 = p.offsets[e] + (chunk - prefix[e]) * kW4MaxTokens;
    it->rows = min(kW4MaxTokens, (int)p.offsets[e + 1] - it->r0);
    it->unit = group * WR;
    // a row block past the last repeats it; its results are not stored
    const int u = it->unit + wu;
    const int rb0 = min(kGated ? u : 2 * u, rb_n - 1), rb1 = kGated ? rb0 : min(2 * u + 1, rb_n - 1);
    it->block[0] = ((long long)e * rb_n + rb0) * sp_n;
    it->block[1] = ((long long)e * rb_n + rb1) * sp_n;
  };
  W4Item cur, nxt;
  place((int)(first / groups), (int)(first % groups), &cur);
  W4Step<GPS> buf[kW4Depth];
#pragma unroll
  for (int b = 0; b < kW4Depth; ++b)
    if (b < n_steps) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const long long blk = cur.block[m] + ks + b * WK;
        const uint8_t* q = p.q[kGated ? m : 0] + blk * kW4Block + lane * 16;
        const __nv_bfloat16* s = p.s[kGated ? m : 0] + (blk * kW4Rows + g) * GPS;
        buf[b].q[m][0] = w4_load_codes(q);
        buf[b].q[m][1] = w4_load_codes(q + kW4Block / 2);
        buf[b].s[m][0].load(s);
        buf[b].s[m][1].load(s + 8 * GPS);
      }
    }
  int flip = 0;
  for (long long i = first; i < end; ++i) {
    if (i + 1 < end) {
      const bool wrap = cur.group + 1 == groups;
      place(cur.chunk + wrap, wrap ? 0 : cur.group + 1, &nxt);
    } else {
      nxt = cur;
      nxt.rows = 0;
    }
    const int nt = (cur.rows + 7) / 8;
    float4* r = red + (nt <= 2 && flip ? kW4Warps * 2 * 2 * 32 : 0);
    if (nt > 2) __syncthreads();  // the last item's sums are still being read
    switch (nt) {
      case 1: w4_item<1, GPS, kGated, WR>(p, cur, nxt, n_steps, buf, r); break;
      case 2: w4_item<2, GPS, kGated, WR>(p, cur, nxt, n_steps, buf, r); break;
      case 3: w4_item<3, GPS, kGated, WR>(p, cur, nxt, n_steps, buf, r); break;
      default: w4_item<4, GPS, kGated, WR>(p, cur, nxt, n_steps, buf, r); break;
    }
    // sums of more than two tiles fill both buffers
    if (nt > 2) __syncthreads();
    flip ^= 1;
    cur = nxt;
  }
}

}  // namespace moe
