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
// expert's codes are streamed once and every other cost has to stay below that
// stream.  The weights are the 16-row operand of mma.m16n8k16 (M = output rows),
// the tokens its 8 columns; up to 4 column tiles (32 rows of an expert) share one
// pass over the codes.
//   * A warp's step is two row blocks x 128 columns (2 KiB of codes).  A lane holds
//     16 bytes of a row: columns 32 j + 8 t .. + 7 for j = 0..3.  The order of a
//     contraction is free, so the instruction's k slots are given the columns as
//     they lie, and the token operand is the matching 16 bytes of the token row.
//   * Codes become bf16 exactly.  A nibble alone in the low eight bits of a bf16 is
//     the subnormal (or first normal) number code * 2^-133 resp. code * 2^-129, so
//     one fused multiply-add with 2^127 resp. 2^123 and -1/8 gives (code - 8) / 64;
//     the 64 joins at the end.  A word of eight codes costs one shift, four ands and
//     four multiply-adds.  Products are exact in fp32; each group's fp32 sum is
//     multiplied by the group's scale in fp32, so the weights are never rounded.
//   * The CTA's eight warps take WR pairs of row blocks times WK = 8 / WR slices of
//     the contraction; slices are joined through shared memory in slice order.
//   * Items (row chunk of an expert, WR pairs of row blocks) are cut into equal
//     contiguous runs, one per CTA.  Codes, scales and token rows come through a ring
//     of shared-memory stages (cp.async), filled D - 1 steps ahead across items; a
//     warp's codes are its own, a token tile is shared by the WR warps of a slice.
// ---------------------------------------------------------------------------
constexpr int kW4Warps = 8;

MOE_DEV uint4 w4_lds(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// The columns (2 i, 2 i + 1) of a code word whose nibbles i and i + 4 lie at bits
// 4 H .. + 3 of both halves, as a packed bf16 pair of (code - 8) / 64.
template <int H>
MOE_DEV uint32_t w4_pair(uint32_t w) {
  const uint32_t v = w & (H ? 0x00f000f0u : 0x000f000fu);
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;"
      : "=r"(r) : "r"(v), "r"(H ? 0x7d007d00u : 0x7f007f00u), "r"(0xbe00be00u));
  return r;
}

MOE_DEV void w4_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the first product of a group: c is only written
MOE_DEV void w4_mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The scales of one row and column block: GPS bf16 values.
template <int GPS> struct W4Scale;
template <> struct W4Scale<1> {
  uint16_t v;
  MOE_DEV void load(const char* p) { v = *reinterpret_cast<const uint16_t*>(p); }
  MOE_DEV float get(int) const { return __uint_as_float((uint32_t)v << 16); }
};
template <> struct W4Scale<2> {
  uint32_t v;
  MOE_DEV void load(const char* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  MOE_DEV float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
};
template <> struct W4Scale<4> {
  uint2 v;
  MOE_DEV void load(const char* p) { v = *reinterpret_cast<const uint2*>(p); }
  MOE_DEV float get(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
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

// Shared memory of one kernel variant.  NT: column tiles of 8 rows per chunk.
template <int GPS, int WR, int NT>
struct W4Cfg {
  static constexpr int kWk = kW4Warps / WR, kRows = 8 * NT;
  static constexpr int kDepth = NT == 1 ? 3 : 4;
  static constexpr int kScaleBytes = 2 * kW4Rows * GPS * 2;     // of a warp's two row blocks
  static constexpr int kCodeStage = 2 * kW4Block + kScaleBytes;
  static constexpr int kXStage = NT * 4 * 512;
  static constexpr int kCodes = kW4Warps * kDepth * kCodeStage;
  static constexpr int kX = kWk * kDepth * kXStage;
  static constexpr int kRed = kWk > 1 ? kW4Warps * 2 * NT * 512 : 0;
  static constexpr int kBytes = kCodes + kX + kRed;
};

// A position in a CTA's run of items: chunk of an expert's rows and group of WR
// pairs of row blocks.
struct W4Cursor {
  int e, chunk, group;
  int r0, rows;  // first routed row of the chunk and how many
  MOE_DEV void rows_of(const W4Problem& p, const int* prefix, int per) {
    r0 = p.offsets[e] + (chunk - prefix[e]) * per;
    rows = min(per, (int)p.offsets[e + 1] - r0);
  }
  MOE_DEV void set(const W4Problem& p, const int* prefix, int per, int c, int g) {
    chunk = c;
    group = g;
    e = find_expert(prefix, p.N, c);
    rows_of(p, prefix, per);
  }
  // to the next item of the run; true: it is of another chunk
  MOE_DEV bool next(const W4Problem& p, const int* prefix, int per, int groups) {
    if (++group < groups) return false;
    group = 0;
    ++chunk;
    while (e + 1 < p.N && prefix[e + 1] <= chunk) ++e;
    rows_of(p, prefix, per);
    return true;
  }
};

// One step's products of a warp's two row blocks with NT column tiles.
template <int GPS, int NT>
MOE_DEV void w4_step(const char* codes, const char* xs, float (&acc)[2][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  constexpr int kPer = 4 / GPS;  // 32-column pieces of one group
  uint4 q[2][2];
  W4Scale<GPS> sc[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      q[m][h] = w4_lds(codes + m * kW4Block + h * (kW4Block / 2) + lane * 16);
      sc[m][h].load(codes + 2 * kW4Block + (m * kW4Rows + h * 8 + g) * (GPS * 2));
    }
  float c[2][NT][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = w4_lds(xs + (n * 4 + j) * 512 + lane * 16);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t lo = j == 0 ? q[m][0].x : j == 1 ? q[m][0].y : j == 2 ? q[m][0].z : q[m][0].w;
      const uint32_t hi = j == 0 ? q[m][1].x : j == 1 ? q[m][1].y : j == 2 ? q[m][1].z : q[m][1].w;
      const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
      const uint32_t a01[4] = {w4_pair<0>(lo), w4_pair<0>(hi), w4_pair<1>(lo), w4_pair<1>(hi)};
      const uint32_t a23[4] = {w4_pair<0>(lo8), w4_pair<0>(hi8), w4_pair<1>(lo8), w4_pair<1>(hi8)};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (j % kPer == 0) w4_mma_first(c[m][n], a01, x[n].x, x[n].y);
        else w4_mma(c[m][n], a01, x[n].x, x[n].y);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) w4_mma(c[m][n], a23, x[n].z, x[n].w);
      if (j % kPer == kPer - 1) {
        const float s0 = sc[m][0].get(j / kPer), s1 = sc[m][1].get(j / kPer);
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

// Stores one 16 x 8 piece of the result: output columns c0, c0 + 8 of rows i0, i0 + 1.
MOE_DEV void w4_store(const W4Problem& p, const W4Cursor& it, int rb, int n, float4 v) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int i0 = n * 8 + 2 * t, c0 = rb * kW4Rows + g;
  __nv_bfloat16* out = p.c + (size_t)(it.r0 + i0) * p.n_out;
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i0 + (k & 1) < it.rows && c0 + (k >> 1) * 8 < p.n_out)
      out[(size_t)(k & 1) * p.n_out + c0 + (k >> 1) * 8] = __float2bfloat16_rn(f[k]);
}

MOE_DEV float4 w4_scaled(const float (&a)[4]) {
  return make_float4(64.f * a[0], 64.f * a[1], 64.f * a[2], 64.f * a[3]);
}
MOE_DEV float4 w4_act(float4 v, float4 up) {
  return make_float4(silu(v.x) * up.x, silu(v.y) * up.y, silu(v.z) * up.z, silu(v.w) * up.w);
}

template <int GPS, bool kGated, int WR, int MaxNT>
struct W4Kernel {
  using Cfg = W4Cfg<GPS, WR, MaxNT>;
  static constexpr int WK = Cfg::kWk, D = Cfg::kDepth;
  // token pieces (column tile, 32-column piece) that a warp copies per stage, and the
  // column tiles among them
  static constexpr int kPieces = MaxNT * 4 >= WR ? MaxNT * 4 / WR : 1;
  static constexpr int kTiles = WR == 8 ? (MaxNT + 1) / 2 : MaxNT;

  const W4Problem& p;
  const int* prefix;
  char *codes, *xs;  // this warp's and this slice's ring
  float4* red;
  int rb_n, sp_n, groups, n_steps, ks, wu;
  W4Cursor load;
  int load_step, load_slot, slot;
  long long load_left;   // items of the run that are not loaded yet
  int xrow[kTiles];

  MOE_DEV int row_block(int group, int m) const {
    const int u = group * WR + wu;
    // a row block past the last repeats it; its results are not stored
    return min(kGated ? u : 2 * u + m, rb_n - 1);
  }
  MOE_DEV int tile_of(int i) const { return WR == 8 ? 2 * i + (wu >> 2) : i; }

  // The token rows that this lane copies of the load cursor's chunk.
  MOE_DEV void take_rows() {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int r = tile_of(i) * 8 + g;
      xrow[i] = 0;
      if (r < load.rows) {
        xrow[i] = load.r0 + r;
        if (p.a_rows) {
          xrow[i] = p.a_rows[load.r0 + r];
          if (xrow[i] < 0 || xrow[i] >= p.a_src_rows) {
            set_status(p.status, MOE_DEV_BAD_OFFSETS);
            xrow[i] = 0;
          }
        }
      }
    }
  }

  // Issues the copies of the load cursor's step and moves it on; one group per call.
  MOE_DEV void fill() {
    if (load_left > 0) {
      const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
      const int kb = ks + load_step * WK;
      char* dst = codes + load_slot * Cfg::kCodeStage;
      long long blk[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        blk[m] = ((long long)load.e * rb_n + row_block(load.group, m)) * sp_n + kb;
        const uint8_t* q = p.q[kGated ? m : 0] + blk[m] * kW4Block + lane * 16;
        cp_async16(dst + m * kW4Block + lane * 16, q);
        cp_async16(dst + m * kW4Block + kW4Block / 2 + lane * 16, q + kW4Block / 2);
      }
      constexpr int kEach = GPS == 4 ? 8 : 4, kHalf = Cfg::kScaleBytes / 2 / kEach;  // lanes per block
      if (lane < 2 * kHalf) {
        const int m = lane / kHalf;
        const char* s = reinterpret_cast<const char*>(p.s[kGated ? m : 0]) +
                        (m ? blk[1] : blk[0]) * (kW4Rows * GPS * 2) + (lane % kHalf) * kEach;
        cp_async_small<kEach>(dst + 2 * kW4Block + lane * kEach, s);
      }
      char* xd = xs + load_slot * Cfg::kXStage + lane * 16;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int piece = wu + i * WR, n = piece >> 2, j = piece & 3;
        const int row = xrow[WR == 8 ? i : WR == 4 ? i : WR == 2 ? i / 2 : i / 4];
        const int k = kb * kW4Cols + 32 * j + 8 * t;
        if (piece < MaxNT * 4 && n * 8 + g < load.rows) {
          if (k < p.k_dim) cp_async16(xd + piece * 512, p.a + (size_t)row * p.k_dim + k);
          else *reinterpret_cast<uint4*>(xd + piece * 512) = make_uint4(0, 0, 0, 0);
        }
      }
      load_slot = load_slot + 1 == D ? 0 : load_slot + 1;
      if (++load_step == n_steps) {
        load_step = 0;
        if (--load_left > 0 && load.next(p, prefix, Cfg::kRows, groups)) take_rows();
      }
    }
    cp_async_commit();
  }

  // The WR warps of a slice.
  MOE_DEV void slice_sync() {
    if constexpr (WR == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + ks), "n"(WR * 32) : "memory");
  }

  template <int NT>
  MOE_DEV void item(const W4Cursor& it) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][n][k] = 0.f;
    for (int i = 0; i < n_steps; ++i) {
      cp_async_wait<D - 2>();
      slice_sync();  // every copy of this stage has landed, the stage before is read
      fill();
      w4_step<GPS, NT>(codes + slot * Cfg::kCodeStage, xs + slot * Cfg::kXStage, acc);
      slot = slot + 1 == D ? 0 : slot + 1;
    }
    if constexpr (WK == 1) {
      const int u = it.group * WR + wu;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (kGated) {
          if (u < rb_n) w4_store(p, it, u, n, w4_act(w4_scaled(acc[0][n]), w4_scaled(acc[1][n])));
        } else {
#pragma unroll
          for (int m = 0; m < 2; ++m)
            if (2 * u + m < rb_n) w4_store(p, it, 2 * u + m, n, w4_scaled(acc[m][n]));
        }
      }
    } else {
      // join the slices: slot (warp, row block, column tile) of 32 lanes
      __syncthreads();  // the last item's sums have been read
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          red[((warp * 2 + m) * NT + n) * 32 + lane] = w4_scaled(acc[m][n]);
      __syncthreads();
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
        if (kGated) v = w4_act(v, join(1));
        const int rb = kGated ? it.group * WR + u : 2 * (it.group * WR + u) + m;
        if (rb < rb_n) w4_store(p, it, rb, n, v);
      }
    }
  }
};

template <int GPS, bool kGated, int WR, int MaxNT>
__global__ void __launch_bounds__(kW4Warps * 32, 2)
w4_mma_kernel(const __grid_constant__ W4Problem p) {
  pdl_trigger();
  pdl_wait();
  using K = W4Kernel<GPS, kGated, WR, MaxNT>;
  using Cfg = typename K::Cfg;
  constexpr int WK = Cfg::kWk;
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int scan_tmp[33];
  extern __shared__ __align__(16) char w4_smem[];
  build_chunk_prefix(p.offsets, p.N, p.max_rows, Cfg::kRows, prefix, scan_tmp, p.status);
  const int rb_n = w4_row_blocks(p.n_out), sp_n = w4_col_blocks(p.k_dim);
  const int units = kGated ? rb_n : (rb_n + 1) / 2;
  const int groups = (units + WR - 1) / WR;
  const long long total = (long long)prefix[p.N] * groups;
  const long long first = total * blockIdx.x / gridDim.x;
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  if (first >= end) return;
  const int warp = threadIdx.x >> 5, ks = warp % WK;
  K k{p, prefix, w4_smem + warp * Cfg::kDepth * Cfg::kCodeStage,
      w4_smem + Cfg::kCodes + ks * Cfg::kDepth * Cfg::kXStage,
      reinterpret_cast<float4*>(w4_smem + Cfg::kCodes + Cfg::kX)};
  k.rb_n = rb_n;
  k.sp_n = sp_n;
  k.groups = groups;
  k.ks = ks;
  k.wu = warp / WK;
  k.n_steps = sp_n > ks ? (sp_n - ks + WK - 1) / WK : 0;
  W4Cursor cur;
  cur.set(p, prefix, Cfg::kRows, (int)(first / groups), (int)(first % groups));
  k.load = cur;
  k.load_step = k.load_slot = k.slot = 0;
  k.load_left = k.n_steps > 0 ? end - first : 0;
  k.take_rows();
#pragma unroll
  for (int i = 0; i < Cfg::kDepth - 1; ++i) k.fill();
  for (long long i = first;;) {
    const int nt = (cur.rows + 7) / 8;
    if (MaxNT == 1 || nt <= 1) k.template item<1>(cur);
    else if (MaxNT >= 2 && nt == 2) k.template item<MaxNT >= 2 ? 2 : 1>(cur);
    else if (MaxNT >= 3 && nt == 3) k.template item<MaxNT >= 3 ? 3 : 1>(cur);
    else if (MaxNT >= 4) k.template item<MaxNT >= 4 ? 4 : 1>(cur);
    if (++i >= end) break;
    cur.next(p, prefix, Cfg::kRows, groups);
  }
}

}  // namespace moe
