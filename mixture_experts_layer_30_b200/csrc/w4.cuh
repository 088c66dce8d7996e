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

#include <type_traits>

#include "common.cuh"

namespace moe {

constexpr int kW4Rows = 16, kW4Cols = 128, kW4Block = 1024;  // one block of codes, bytes

// unsigned: the rounding up of a size next to 2^31
__host__ MOE_DEV int w4_row_blocks(int rows) { return ((unsigned)rows + kW4Rows - 1) / kW4Rows; }
__host__ MOE_DEV int w4_col_blocks(int cols) { return ((unsigned)cols + kW4Cols - 1) / kW4Cols; }

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
// the tokens its 8 columns; up to 2 column tiles (16 rows of an expert) share one
// pass over the codes.  Bound by instruction issue: a step below takes 280 to 340
// instructions a warp, 144 of them to decode, and four warps a scheduler reach 0.6 of
// the issue rate.  Down product at d = 6144, I = 2048, N = 32, 13 tokens, groups of 32:
// 47 to 49 us, 4.4 to 4.5 TB/s by the codes, scales and rows of the 30 experts that have
// any; gate/up of the mid layer (64 x 2048 x 1024) at 256 tokens, groups of 64: 59 us,
// 1.9 TB/s (49 experts).  The same products on tcgen05 (codes decoded into tensor memory,
// the groups' sums read back for their scales) took longer up to 24 rows an expert: 60
// against 48 us at 16 rows; a half step's chain of store, barrier, products and sums is
// longer than its decoding.
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
//     the contraction; the warps of a pair join their slices through shared memory in
//     slice order.
//   * Items (row chunk of an expert, WR pairs of row blocks) are cut into contiguous
//     runs of equal cost, one per CTA.  Codes and scales come through a ring of
//     shared-memory stages (cp.async) filled two steps ahead across items, token rows
//     (from L2) one step ahead; a warp's codes are its own, a token tile is shared by
//     the WR warps of a slice.  A third resident CTA with shorter rings was slower (77
//     against 57 us at 256 tokens of the mid layer), a deeper ring not faster.
// ---------------------------------------------------------------------------
constexpr int kW4Warps = 8;

// (Loads are ordered by the "memory" clobbers of the waits and barriers around a step.)
template <int kOffset>
MOE_DEV uint4 w4_lds(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at), "n"(kOffset));
  return v;
}

// (a, b) += s * (x, y) as one instruction on pairs.
MOE_DEV void w4_fma2(float& a, float& b, uint64_t s, float x, float y) {
  f2_unpack(f2_fma(s, f2_pack(x, y), f2_pack(a, b)), a, b);
}

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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the first product of a group: c is only written
MOE_DEV void w4_mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The scales of one row and column block: GPS bf16 values.
template <int GPS> struct W4Scale;
template <> struct W4Scale<1> {
  uint16_t v;
  template <int kOffset> MOE_DEV void load(uint32_t at) {
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v) : "r"(at), "n"(kOffset));
  }
  MOE_DEV float get(int) const { return __uint_as_float((uint32_t)v << 16); }
};
template <> struct W4Scale<2> {
  uint32_t v;
  template <int kOffset> MOE_DEV void load(uint32_t at) {
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(v) : "r"(at), "n"(kOffset));
  }
  MOE_DEV float get(int i) const { return __uint_as_float(i ? v & 0xffff0000u : v << 16); }
};
template <> struct W4Scale<4> {
  uint32_t v[2];
  template <int kOffset> MOE_DEV void load(uint32_t at) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];"
                 : "=r"(v[0]), "=r"(v[1]) : "r"(at), "n"(kOffset));
  }
  MOE_DEV float get(int i) const {
    return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
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

// One kernel variant.  NT: column tiles of 8 rows per chunk.
template <int GPS, int WR, int NT>
struct W4Cfg {
  static_assert(WR >= NT, "a warp copies pieces of one column tile");
  static_assert(WR < kW4Warps, "the warps of a pair join slices");
  static constexpr int kWk = kW4Warps / WR, kRows = 8 * NT;
  static constexpr int kDepth = 3;
  static constexpr int kScaleBytes = 2 * kW4Rows * GPS * 2;     // of a warp's two row blocks
  static constexpr int kCodeStage = 2 * kW4Block + kScaleBytes;
  static constexpr int kXStage = NT * 4 * 512;
  static constexpr int kCodes = kW4Warps * kDepth * kCodeStage;
  static constexpr int kX = kWk * 2 * kXStage;
  static constexpr int kRed = (kWk - 1) * WR * 2 * NT * 512;
  static constexpr int kBytes = kCodes + kX + kRed;  // and two tables of N + 1 and 33 ints
  // Cost of a chunk: 8 rows against 16 an expert take 35 and 44 us for the mid layer's
  // gate/up (64 experts, 2048 x 1024, groups of 128), of which about 5 are the call's.
  static MOE_DEV int weight(int rows) { return NT == 1 ? 1 : rows <= 8 ? 5 : 6; }
};

// An item: WR pairs of row blocks (group) for one chunk of an expert's rows.
template <typename Cfg>
struct W4Cursor {
  int e, c, group;
  int r0, rows;  // first routed row of the chunk and how many
  MOE_DEV void take(const int* off) {
    r0 = off[e] + c * Cfg::kRows;
    rows = min(Cfg::kRows, off[e + 1] - r0);
  }
  // Behind the expert's last chunk: to the next expert that has rows (or to N).
  MOE_DEV void settle(const int* off, const int* cost, int N) {
    if (off[e] + c * Cfg::kRows < off[e + 1]) return;
    c = 0;
    do ++e;
    while (e < N && cost[e + 1] == cost[e]);
  }
  // The first item that starts at or behind part / parts of all costs (U holds their product
  // with parts: 32 bits where they do, for the divisions' latency).
  template <typename U>
  MOE_DEV void seek(const int* off, const int* cost, int N, int groups, int part, int parts) {
    const U at = (U)cost[N] * groups * part / parts;
    c = group = 0;
    e = N;
    if (part == parts || at >= (U)cost[N] * groups) return;
    e = find_expert(cost, N, (int)(at / groups));
    U rem = at - (U)cost[e] * groups;
    const U full = (U)Cfg::weight(Cfg::kRows) * groups;
    const int last = (off[e + 1] - off[e] - 1) / Cfg::kRows;
    if (last > 0) c = (int)min(rem / full, (U)last);
    rem -= c * full;
    take(off);
    const int w = Cfg::weight(rows);
    group = (int)((rem + w - 1) / w);
    if (group >= groups) {
      group = 0;
      ++c;
      settle(off, cost, N);
    }
  }
  // To the next item; true: it is of another chunk.
  MOE_DEV bool next(const int* off, const int* cost, int N, int groups) {
    if (++group < groups) return false;
    group = 0;
    ++c;
    settle(off, cost, N);
    return true;
  }
  MOE_DEV bool same(const W4Cursor& o) const { return e == o.e && c == o.c && group == o.group; }
};

// cost[e] = sum of the weights of experts 0..e-1's chunks, off[] = offsets; segments that
// are not ascending or out of range count as empty and are reported.  Ends with a barrier.
template <typename Cfg>
MOE_DEV void w4_costs(const W4Problem& p, int* off, int* cost, int* scan_tmp) {
  const int per = (p.N + blockDim.x - 1) / blockDim.x;
  const int lo = min(p.N, (int)threadIdx.x * per), hi = min(p.N, lo + per);
  auto weigh = [&](int e, bool report) {
    const int a = p.offsets[e], b = p.offsets[e + 1], m = b - a;
    if (report) off[e] = a;
    if (m < 0 || a < 0 || b > p.max_rows) {
      if (report) set_status(p.status, MOE_DEV_BAD_OFFSETS);
      return 0;
    }
    const int full = m / Cfg::kRows, rest = m % Cfg::kRows;
    return full * Cfg::weight(Cfg::kRows) + (rest ? Cfg::weight(rest) : 0);
  };
  int local = 0;
  for (int e = lo; e < hi; ++e) local += weigh(e, true);
  int run = block_exclusive_scan(local, scan_tmp, &scan_tmp[32]);
  for (int e = lo; e < hi; ++e) {
    cost[e] = run;
    if (per > 1) run += weigh(e, false);
  }
  if (threadIdx.x == 0) {
    cost[p.N] = scan_tmp[32];
    off[p.N] = p.offsets[p.N];
  }
  __syncthreads();
}

// One step's products of a warp's two row blocks with NT column tiles.  codes, x: this
// lane's 16 bytes of the first row half resp. token piece, scales: its row's.  kPairs: the
// scaled sums two at a time (with several column tiles the pairs' registers cost more).
template <int GPS, int NT, bool kPairs>
MOE_DEV void w4_step(uint32_t codes, uint32_t scales, uint32_t xs, float (&acc)[2][NT][4]) {
  constexpr int kPer = 4 / GPS;  // 32-column pieces of one group
  constexpr int kHalfScales = 8 * GPS * 2;
  uint4 q[2][2];
  W4Scale<GPS> sc[2][2];
  q[0][0] = w4_lds<0>(codes);
  q[0][1] = w4_lds<kW4Block / 2>(codes);
  q[1][0] = w4_lds<kW4Block>(codes);
  q[1][1] = w4_lds<kW4Block * 3 / 2>(codes);
  sc[0][0].template load<0>(scales);
  sc[0][1].template load<kHalfScales>(scales);
  sc[1][0].template load<2 * kHalfScales>(scales);
  sc[1][1].template load<3 * kHalfScales>(scales);
  float c[2][NT][4];
  auto piece = [&](auto jc) {
    constexpr int j = decltype(jc)::value;
    uint4 x[NT];
    x[0] = w4_lds<j * 512>(xs);
    if constexpr (NT > 1) x[1] = w4_lds<(4 + j) * 512>(xs);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t lo = j == 0 ? q[m][0].x : j == 1 ? q[m][0].y : j == 2 ? q[m][0].z : q[m][0].w;
      const uint32_t hi = j == 0 ? q[m][1].x : j == 1 ? q[m][1].y : j == 2 ? q[m][1].z : q[m][1].w;
      const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
      const uint32_t a01[4] = {w4_pair<0>(lo), w4_pair<0>(hi), w4_pair<1>(lo), w4_pair<1>(hi)};
      const uint32_t a23[4] = {w4_pair<0>(lo8), w4_pair<0>(hi8), w4_pair<1>(lo8), w4_pair<1>(hi8)};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (j % kPer == 0) w4_mma_first(c[m][n], a01, x[n].x, x[n].y);
        else w4_mma(c[m][n], a01, x[n].x, x[n].y);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) w4_mma(c[m][n], a23, x[n].z, x[n].w);
      if constexpr (j % kPer == kPer - 1) {
        const float f0 = sc[m][0].get(j / kPer), f1 = sc[m][1].get(j / kPer);
        if constexpr (kPairs) {
          const uint64_t s0 = f2_pack(f0, f0), s1 = f2_pack(f1, f1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            w4_fma2(acc[m][n][0], acc[m][n][1], s0, c[m][n][0], c[m][n][1]);
            w4_fma2(acc[m][n][2], acc[m][n][3], s1, c[m][n][2], c[m][n][3]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[m][n][0] = fmaf(f0, c[m][n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(f0, c[m][n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(f1, c[m][n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(f1, c[m][n][3], acc[m][n][3]);
          }
        }
      }
    }
  };
  piece(std::integral_constant<int, 0>{});
  piece(std::integral_constant<int, 1>{});
  piece(std::integral_constant<int, 2>{});
  piece(std::integral_constant<int, 3>{});
}

// Stores one 16 x 8 piece of the result: output columns c0, c0 + 8 of rows i0, i0 + 1.
MOE_DEV void w4_store(const W4Problem& p, int r0, int rows, int rb, int n, float4 v) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int i0 = n * 8 + 2 * t, c0 = rb * kW4Rows + g;
  __nv_bfloat16* out = p.c + (size_t)(r0 + i0) * p.n_out;
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i0 + (k & 1) < rows && c0 + (k >> 1) * 8 < p.n_out)
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
  using Cursor = W4Cursor<Cfg>;
  static constexpr int WK = Cfg::kWk, D = Cfg::kDepth;
  static constexpr int kPieces = 4 * MaxNT / WR;  // 32-column pieces a warp copies per token tile
  static constexpr int kEach = GPS == 4 ? 8 : 4;  // bytes of scales a lane copies
  static constexpr int kHalf = Cfg::kScaleBytes / 2 / kEach;  // lanes of one block's scales

  const W4Problem& p;
  const int *off, *cost;
  float4* red;       // this pair's
  int rb_n, sp_n, groups, n_steps, ks, wu;
  // codes: items and steps of the current one that are not copied yet, this lane's next
  // addresses and where they go (a position of this warp's ring)
  Cursor load;
  int load_left, load_todo;
  const uint8_t *qa, *qb;
  const char* sc;
  uint32_t ring, ring_end, wr;
  uint32_t sc_lane;  // from this lane's codes of a stage to its share of the scales
  // token rows: the same, one step ahead of the products
  Cursor xload;
  int x_left, x_todo, x_cols;  // x_cols: columns of k_dim from this lane's on
  bool x_on;                   // this lane's row exists
  const __nv_bfloat16* xp;
  uint32_t x_piece;            // where its first piece goes in a buffer
  uint32_t rd, x_rd, x_both;   // the products' ring position and buffer; both buffers' sum

  // A row block past the last repeats it; its results are not stored.
  MOE_DEV int row_block(int group, int m) const {
    const int u = group * WR + wu;
    return min(kGated ? u : 2 * u + m, rb_n - 1);
  }
  MOE_DEV void code_item() {
    const int lane = threadIdx.x & 31;
    long long blk[2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
      blk[m] = ((long long)load.e * rb_n + row_block(load.group, m)) * sp_n + ks;
    qa = p.q[0] + blk[0] * kW4Block + lane * 16;
    qb = p.q[kGated ? 1 : 0] + blk[1] * kW4Block + lane * 16;
    const int m = lane / kHalf & 1;
    sc = reinterpret_cast<const char*>(m && kGated ? p.s[1] : p.s[0]) +
         (m ? blk[1] : blk[0]) * (kW4Rows * GPS * 2) + (lane % kHalf) * kEach;
    load_todo = n_steps;
  }
  MOE_DEV void fill_codes() {
    if (load_left > 0) {
      cp_async16(wr, qa);
      cp_async16(wr + kW4Block / 2, qa + kW4Block / 2);
      cp_async16(wr + kW4Block, qb);
      cp_async16(wr + kW4Block * 3 / 2, qb + kW4Block / 2);
      if (2 * kHalf == 32 || (threadIdx.x & 31) < 2 * kHalf) cp_async_small<kEach>(wr + sc_lane, sc);
      qa += WK * kW4Block;
      qb += WK * kW4Block;
      sc += WK * kW4Rows * GPS * 2;
      wr += Cfg::kCodeStage;
      if (wr >= ring_end) wr -= D * Cfg::kCodeStage;
      if (--load_todo == 0 && --load_left > 0) {
        load.next(off, cost, p.N, groups);
        code_item();
      }
    }
    cp_async_commit();
  }

  // This lane's part of the chunk's token rows: row g of column tile wu / (WR / MaxNT), the
  // pieces from wu % (WR / MaxNT) * kPieces on, eight columns t of each.
  MOE_DEV void x_item(bool rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int col = ks * kW4Cols + wu % (WR / MaxNT) * kPieces * 32 + 8 * t;
    if (rows) {
      const int r = wu / (WR / MaxNT) * 8 + g;
      int row = 0;
      x_on = r < xload.rows;
      if (x_on) {
        row = xload.r0 + r;
        if (p.a_rows) {
          row = p.a_rows[row];
          if (row < 0 || row >= p.a_src_rows) {
            set_status(p.status, MOE_DEV_BAD_OFFSETS);
            row = 0;
          }
        }
      }
      xp = p.a + (size_t)row * p.k_dim + col;
    } else {
      xp -= n_steps * WK * kW4Cols;
    }
    x_cols = p.k_dim - col;
    x_todo = n_steps;
  }
  MOE_DEV void fill_x(uint32_t buffer) {
    if (x_left > 0) {
      if (x_on) {
        const uint32_t dst = buffer + x_piece;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          cp_async16_or_zero(dst + j * 512, xp + 32 * j, x_cols > 32 * j);
        }
      }
      xp += WK * kW4Cols;
      x_cols -= WK * kW4Cols;
      if (--x_todo == 0 && --x_left > 0) {
        const bool rows = xload.next(off, cost, p.N, groups);
        if (rows) xload.take(off);
        x_item(rows);
      }
    }
    cp_async_commit();
  }

  template <int NT>
  MOE_DEV void item(const Cursor& it) {
    const int lane = threadIdx.x & 31;
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][n][k] = 0.f;
    for (int i = 0; i < n_steps; ++i) {
      // all but the newest group, the next step's codes: it was issued behind this step's tokens
      cp_async_wait<1>();
      // every copy of this step has landed, and the step before is read
      asm volatile("bar.sync %0, %1;" ::"r"(1 + ks), "n"(WR * 32) : "memory");
      const uint32_t other = x_both - x_rd;
      fill_x(other);
      fill_codes();
      w4_step<GPS, NT, MaxNT == 1 || GPS != 1>(rd + lane * 16, rd + 2 * kW4Block + (lane >> 2) * (GPS * 2), x_rd, acc);
      rd += Cfg::kCodeStage;
      if (rd >= ring_end) rd -= D * Cfg::kCodeStage;
      x_rd = other;
    }
    auto store = [&](int n, float4 v0, float4 v1) {
      const int u = it.group * WR + wu;
      if constexpr (kGated) {
        if (u < rb_n) w4_store(p, it.r0, it.rows, u, n, w4_act(v0, v1));
      } else {
        if (2 * u < rb_n) w4_store(p, it.r0, it.rows, 2 * u, n, v0);
        if (2 * u + 1 < rb_n) w4_store(p, it.r0, it.rows, 2 * u + 1, n, v1);
      }
    };
    // slices 1.. leave their sums to slice 0, which adds them in slice order
    auto pair_sync = [&] {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + WK + wu), "n"(WK * 32) : "memory");
    };
    pair_sync();  // the last item's sums have been read
    if (ks > 0) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          red[(((ks - 1) * 2 + m) * NT + n) * 32 + lane] = w4_scaled(acc[m][n]);
    }
    pair_sync();
    if (ks == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float4 v[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          v[m] = w4_scaled(acc[m][n]);
#pragma unroll
          for (int k = 0; k < WK - 1; ++k) {
            const float4 w = red[((k * 2 + m) * NT + n) * 32 + lane];
            v[m].x += w.x;
            v[m].y += w.y;
            v[m].z += w.z;
            v[m].w += w.w;
          }
        }
        store(n, v[0], v[1]);
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
  extern __shared__ __align__(16) char w4_smem[];
  int* off = reinterpret_cast<int*>(w4_smem + Cfg::kBytes);
  int* cost = off + p.N + 1;
  w4_costs<Cfg>(p, off, cost, cost + p.N + 1);
  const int rb_n = w4_row_blocks(p.n_out), sp_n = w4_col_blocks(p.k_dim);
  const int units = kGated ? rb_n : (rb_n + 1) / 2;
  const int groups = (units + WR - 1) / WR;
  // even lanes look for the start of this CTA's run, odd ones for its end
  typename K::Cursor cur, end;
  const int part = blockIdx.x + (threadIdx.x & 1);
  if ((long long)cost[p.N] * groups * gridDim.x < (1LL << 32))
    end.template seek<uint32_t>(off, cost, p.N, groups, part, gridDim.x);
  else
    end.template seek<unsigned long long>(off, cost, p.N, groups, part, gridDim.x);
  auto from = [](int v, int lane) { return __shfl_sync(0xffffffffu, v, lane); };
  cur.e = from(end.e, 0);
  cur.c = from(end.c, 0);
  cur.group = from(end.group, 0);
  end.e = from(end.e, 1);
  end.c = from(end.c, 1);
  end.group = from(end.group, 1);
  int left = 0;
  for (typename K::Cursor c = cur; !c.same(end); ++left) c.next(off, cost, p.N, groups);
  if (left == 0) return;
  cur.take(off);
  const int warp = threadIdx.x >> 5, ks = warp % WK, wu = warp / WK;
  const int lane = threadIdx.x & 31;
  K k{p, off, cost,
      reinterpret_cast<float4*>(w4_smem + Cfg::kCodes + Cfg::kX + wu * (Cfg::kRed / WR))};
  k.rb_n = rb_n;
  k.sp_n = sp_n;
  k.groups = groups;
  k.ks = ks;
  k.wu = wu;
  k.n_steps = sp_n > ks ? (sp_n - ks + WK - 1) / WK : 0;
  k.rd = smem_at(w4_smem) + warp * Cfg::kDepth * Cfg::kCodeStage;
  k.ring_end = k.rd + Cfg::kDepth * Cfg::kCodeStage;
  k.wr = k.rd + lane * 16;
  k.sc_lane = 2 * kW4Block + lane * K::kEach - lane * 16;
  const uint32_t xbuf = smem_at(w4_smem) + Cfg::kCodes + ks * 2 * Cfg::kXStage + lane * 16;
  k.x_piece = (wu / (WR / MaxNT) * 4 + wu % (WR / MaxNT) * K::kPieces) * 512;
  k.x_rd = xbuf;
  k.x_both = 2 * xbuf + Cfg::kXStage;
  k.load = k.xload = cur;
  k.load_left = k.x_left = k.n_steps > 0 ? left : 0;
  k.code_item();
#pragma unroll
  for (int i = 0; i < Cfg::kDepth - 2; ++i) k.fill_codes();
  k.x_item(true);
  k.fill_x(xbuf);
  k.fill_codes();
  for (;;) {
    const int nt = (cur.rows + 7) / 8;
    if (nt <= 1) k.template item<1>(cur);
    else k.template item<MaxNT>(cur);
    if (--left == 0) break;
    if (cur.next(off, cost, p.N, groups)) cur.take(off);
  }
}

}  // namespace moe
