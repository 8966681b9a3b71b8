// Warp-level building blocks for one tile of 8-bit codes (S keys x D dims, one
// byte an element) in shared memory, against the query heads of a group:
//
//   scores: S^T (S keys x columns) = X_tile (keys x D) . Q^T (D x columns)
//   values: O^T (D x columns)      = Y_tile^T (D x keys) . P^T (keys x columns)
//
// Two sets of the same functions, both exact in the codes:
//
// * HalfOps: m16n8k16 in half precision, which holds every code of either format
//   exactly (int8: integers up to 128; e4m3: four significant bits, 2^-9 .. 448),
//   eight heads in the eight columns.  A query row is scaled by a power of two so
//   that its largest element is in [2^14, 2^15): bf16's 8 bits fit half
//   precision's 11, down to elements 2^-28 of the largest.  Weights e^{x - max}
//   are computed times 2^15 for the same reason: within 2^-11 of themselves, or
//   2^-40 of the largest.  PARTS = 2 (float32 configurations) holds queries and
//   weights as a sum of two halves (the nearest one and the rest): within 2^-22.
//   bf16 configurations take one half of a weight: their results round to bf16, 2^-8
//   of themselves, and over e4m3 codes are off by 1.665e-3 (2-norm, against 64
//   bits) where plain 32-bit arithmetic is by 1.657e-3.  A second half makes it
//   1.657e-3 and takes 7% longer (attention, 96 x 16K: 84.3 -> 90.4 us), 15% for
//   summaries (128K tokens: 37.1 -> 42.7).
// * DigitOps (int8 codes, bf16, up to four heads): 8-bit m16n8k32 with int32 sums
//   on the codes as they are.  A query or weight is a fixed-point number in 8-bit
//   digits, each a column of its own: three for a query (within 2^-24 of its
//   row's largest element: scores and entropies keep float32's accuracy), two
//   for a weight (within 2^-16 of the largest), which only enters a result that
//   rounds to bf16 (2^-8).
// The sum of the weights is always taken in float32 from the unrounded ones.
//
// Which: widening costs an int8 code five instructions for four codes on the
// pipe that limits, an e4m3 code two or three.  DigitOps : HalfOps, us: decode
// attention over int8, 64 sequences of 16K (K = 32, W = 512), G = 1 56.9 : 60.5,
// G = 4 58.2 : 62.4; summaries of 55K tokens, G = 2, 18.1 : 24.5.  Eight heads need
// two blocks of columns: 92.4 : 67.7.  e4m3 digits (two e4m3 numbers): attention
// at G = 1, 4, 8 70.6 : 66.0, 72.5 : 71.0, 96.1 : 73.0, and weights to 2^-8 only.
//
// The tile is stored in lines of 128 bytes whose 16-byte pieces are swizzled as
// TMA does (piece i of line r at i ^ (r & 7)); with gq = lane / 4, c4 = lane % 4:
// * scores: the contraction index is permuted, alike for X and Q: thread c4 holds
//   the D / 4 dims from c4 D / 4 on, in words of four codes.  The eight lanes of
//   one of a load's phases touch all eight pieces of a line once.  Result
//   sc[r][2 mt + hi]: key 16 mt + gq + 8 hi, head head(r, c4).
// * values: a thread holds dims gq D / 8 + x, x < D / 8: result o[r][x]; half_read()
//   is called once what the thread read of the tile's first half has been used.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace hils {

HILS_DI uint32_t movmatrix_trans16(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col)
HILS_DI void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D(16x8, s32) += A(16x32, s8, row) * B(32x8, s8, col)
HILS_DI void mma_8bit(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same without a D to add to
HILS_DI void mma_f16_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
HILS_DI void mma_8bit_first(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
}
HILS_DI uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// the rest of (lo, hi) after pack_f16x2
HILS_DI uint32_t rest_f16x2(float lo, float hi, uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f16x2(lo - f.x, hi - f.y);
}
// 2^x (0 for -inf and wherever 2^x is below the normal range)
HILS_DI float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
HILS_DI float exp_neg(float x) { return exp2_fast(x * kLog2e); }

// byte offset of linear byte `o` of a tile
HILS_DI int swz(int o) { return o ^ (((o >> 7) & 7) << 4); }
// A tile in two halves of S / 2 keys.
template <int D, int S>
struct Tile {
  const uint8_t* h[2];
  // the 16 keys of m-tile mt
  HILS_DI const uint8_t* keys16(int mt) const {
    constexpr int M = S / 32;
    return (mt < M ? h[0] : h[1]) + 16 * (mt < M ? mt : mt - M) * D;
  }
};

// Offsets of a thread's parts in a tile; the pattern repeats every 16 keys.
template <int D>
struct TileOffsets {
  static constexpr int V = D / 64;  // 16-byte pieces of a thread's dims of a key (scores)
  int k[V][2];                      // piece v of key gq + 8 hi
  int v[4];                         // keys 2 c4, + 1, + 8, + 9 (values)
  HILS_DI TileOffsets(int gq, int c4) {
#pragma unroll
    for (int x = 0; x < V; ++x)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) k[x][hi] = swz((gq + 8 * hi) * D + c4 * (D / 4) + 16 * x);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = swz((2 * c4 + (e & 1) + 8 * (e >> 1)) * D + gq * (D / 8));
  }
};

// ------------------------------------------------------------------- codes ---
// Two halves from two codes.  int8: a byte u = code + 128 below 0x64 is the half
// 1024 + u, so subtracting 1152 leaves the code; even and odd bytes of a word
// are taken apart by one mask.  e4m3: the conversion instruction, by half-words.
struct CodeI8 {
  // bytes {0, 2} and {1, 3} of w
  static HILS_DI void halves(uint32_t w, uint32_t& x, uint32_t& y) {
    x = sub((w & 0x00ff00ffu) ^ 0x64806480u);
    y = sub(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u);
  }
  static constexpr int kX1 = 2, kY0 = 1;  // x = (byte 0, byte kX1), y = (byte kY0, byte 3)
  // words of two keys -> (a, b) of bytes 0 and 1 (x), of bytes 2 and 3 (y)
  static HILS_DI uint32_t pair01(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
  static HILS_DI uint32_t pair23(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

  // Digits of x0, x1 in [-kOne, kOne], as bytes lo, hi of x0, then of x1.  Adding
  // 1.5 2^23 + 128 rounds x to an integer in the low bits, where y = x + 128 has
  // hi = y >> 8 and lo = (y & 255) - 128.
  static constexpr float kOne = 32512.f;  // 256 * 127
  static HILS_DI uint32_t digits2(float x0, float x1) {
    const float m = 12582912.f + 128.f;
    return __byte_perm(__float_as_uint(x0 + m), __float_as_uint(x1 + m), 0x5410) ^ 0x00800080u;
  }
  static HILS_DI float join(int hi, int lo) { return (float)(256 * hi + lo); }
  // Queries: integers up to kQuery in three digits, lo, mid, hi in bytes 0 .. 2.
  static constexpr float kQuery = 127.f * 65536.f;
  static HILS_DI void query4(const float (&x)[4], int odd, uint32_t (&w)[2]) {
    uint32_t z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = (uint32_t)(__float2int_rn(x[i]) + 0x8080) ^ 0x8080u;
    const uint32_t s0 = odd ? 0x51u : 0x62u;  // mid : hi
    w[0] = __byte_perm(__byte_perm(z[0], z[1], s0), __byte_perm(z[2], z[3], s0), 0x5410);
    w[1] = odd ? 0u : __byte_perm(__byte_perm(z[0], z[1], 0x40), __byte_perm(z[2], z[3], 0x40), 0x5410);
  }
  static HILS_DI float score(int hi, int mid, int lo) { return fmaf((float)(256 * hi + mid), 256.f, (float)lo); }
  // the factor that brings a row's largest magnitude to kQuery, and its inverse
  static HILS_DI void row_factor(float top, float& down, float& up) {
    top = fmaxf(top, 0x1p-100f);  // smaller ones keep a finite factor
    down = kQuery / top;
    up = top * (1.f / kQuery);
  }
  static constexpr float kLog2One = 14.988684686772166f;

 private:
  static HILS_DI uint32_t sub(uint32_t h) {
    const uint32_t k = 0x64806480u;  // 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
struct CodeE4M3 {
  // bytes {0, 1} and {2, 3} of w
  static HILS_DI void halves(uint32_t w, uint32_t& x, uint32_t& y) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(x), "=r"(y)
        : "r"(w));
  }
  static constexpr int kX1 = 1, kY0 = 2;
  static HILS_DI uint32_t pair01(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5140); }
  static HILS_DI uint32_t pair23(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7362); }
};

// A thread's part of a query row as it is in memory: the D / 4 elements from
// c4 D / 4 on (zeros without a row).
template <typename T, int D>
struct RawRow {
  static constexpr int N = D / 4, PER = 16 / sizeof(T);
  uint4 w[N / PER];
  HILS_DI void load(const T* row, int c4) {
#pragma unroll
    for (int v = 0; v < N / PER; ++v)
      w[v] = row ? __ldg(reinterpret_cast<const uint4*>(row + c4 * N) + v) : make_uint4(0u, 0u, 0u, 0u);
  }
};
// its elements as float32
template <typename T, int D>
HILS_DI void row_values(const RawRow<T, D>& raw, float (&x)[D / 4]) {
  constexpr int PER = 16 / sizeof(T);
#pragma unroll
  for (int v = 0; v < D / 4 / PER; ++v) {
    const uint32_t r[4] = {raw.w[v].x, raw.w[v].y, raw.w[v].z, raw.w[v].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 2) {
        const float2 f = bf16x2_to_f32x2(r[i]);
        x[v * PER + 2 * i] = f.x;
        x[v * PER + 2 * i + 1] = f.y;
      } else {
        x[v * PER + i] = __uint_as_float(r[i]);
      }
    }
  }
}
// over the row's four threads
HILS_DI unsigned row_max(unsigned x) {
  x = max(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return max(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// reductions over the 8 threads that share a column (lanes differing in gq)
HILS_DI float column_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
HILS_DI float column_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// ------------------------------------------------------------- 8-bit products ---
// Column n: head n / 2, digit n & 1; weights (hi, lo); queries (hi, mid), then (lo, none).
template <int D, int S, int G>
struct DigitOps {
  using C = CodeI8;
  static_assert(G <= 4, "one block of columns");
  static_assert(S % 64 == 0, "a half of the tile is read in whole steps of 32 keys");
  static constexpr int R = 1;  // heads of a thread
  static constexpr float kOne = C::kOne, kLog2One = C::kLog2One;  // weights are given times kOne
  static HILS_DI int head(int, int c4) { return c4; }
  static constexpr int Q = 2;
  struct Query {
    uint32_t w[R][Q][D / 16];
    float up[R];  // what a score of head(r, c4) is multiplied by
  };
  // the head whose row a thread gives to make_query
  static HILS_DI int row_head(int gq) { return gq >> 1; }
  template <typename T>
  static HILS_DI void make_query(const RawRow<T, D>& raw, int gq, int c4, Query& q) {
    float x[D / 4], down = 0.f, up = 0.f;
    row_values<T, D>(raw, x);
    unsigned top = 0;  // bits of the largest magnitude, NaN above infinity
#pragma unroll
    for (int i = 0; i < D / 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = row_max(top);
    if (top != 0u && top < 0x7f800000u) C::row_factor(__uint_as_float(top), down, up);
    if (top >= 0x7f800000u) up = __uint_as_float(0x7fc00000u);  // a row with an infinity or NaN scores NaN
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float y[4] = {x[4 * i] * down, x[4 * i + 1] * down, x[4 * i + 2] * down, x[4 * i + 3] * down};
      uint32_t w[Q];
      C::query4(y, gq & 1, w);
#pragma unroll
      for (int d = 0; d < Q; ++d) q.w[0][d][i] = w[d];
    }
    q.up[0] = __shfl_sync(0xffffffffu, up, 8 * c4);
  }
  static HILS_DI void scores(const Tile<D, S>& t, const TileOffsets<D>& at, const Query& q, float (&sc)[R][S / 8]) {
    constexpr int V = D / 64;
#pragma unroll
    for (int mt = 0; mt < S / 16; ++mt) {
      uint32_t w[2][4 * V];
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const uint4 x = *reinterpret_cast<const uint4*>(t.keys16(mt) + at.k[v][hi]);
          w[hi][4 * v] = x.x, w[hi][4 * v + 1] = x.y, w[hi][4 * v + 2] = x.z, w[hi][4 * v + 3] = x.w;
        }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        int d[Q][4];
#pragma unroll
        for (int ks = 0; ks < 2 * V; ++ks) {
          const uint32_t A[4] = {w[0][2 * ks], w[1][2 * ks], w[0][2 * ks + 1], w[1][2 * ks + 1]};
#pragma unroll
          for (int x = 0; x < Q; ++x) {
            if (ks == 0) mma_8bit_first(d[x], A, q.w[r][x][0], q.w[r][x][1]);
            else mma_8bit(d[x], A, q.w[r][x][2 * ks], q.w[r][x][2 * ks + 1]);
          }
        }
        sc[r][2 * mt] = C::score(d[0][0], d[0][1], d[Q - 1][0]);
        sc[r][2 * mt + 1] = C::score(d[0][2], d[0][3], d[Q - 1][2]);
      }
    }
  }
  template <typename F>
  static HILS_DI void values(const Tile<D, S>& t, const TileOffsets<D>& at, int gq, const float (&p)[R][S / 8],
                             float (&o)[R][D / 8], F half_read) {
    // P^T fragments.  A 16-bit element holds the two digits of a weight; the
    // transpose leaves a thread (gq, c4) with head gq / 2 of keys 2 c4 and 2 c4 + 1
    // (+ 8 if gq is odd); it keeps the digit of its column and gets its
    // neighbour's other keys for it.
    uint32_t b[R][S / 16];
    const bool odd = gq & 1;
    const uint32_t keep_s = odd ? 0x6420u : 0x7531u, send_s = odd ? 0x7531u : 0x6420u;
    const uint32_t b0_s = odd ? 0x1054u : 0x5410u, b1_s = odd ? 0x3276u : 0x7632u;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int kk = 0; kk < S / 32; ++kk) {
        const uint32_t x = movmatrix_trans16(C::digits2(p[r][4 * kk], p[r][4 * kk + 1]));
        const uint32_t y = movmatrix_trans16(C::digits2(p[r][4 * kk + 2], p[r][4 * kk + 3]));
        const uint32_t keep = __byte_perm(x, y, keep_s);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, __byte_perm(x, y, send_s), 4);
        b[r][2 * kk] = __byte_perm(keep, got, b0_s);
        b[r][2 * kk + 1] = __byte_perm(keep, got, b1_s);
      }
    constexpr int W = D / 32;  // words of a thread's part of a key
    int d[R][D / 16][4];
#pragma unroll
    for (int kk = 0; kk < S / 32; ++kk) {
      uint32_t w[2][4][W];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint8_t* a = t.keys16(2 * kk + half) + at.v[e];
          if (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(a);
            w[half][e][0] = x.x, w[half][e][1] = x.y, w[half][e][W - 2] = x.z, w[half][e][W - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(a);
            w[half][e][0] = x.x, w[half][e][1] = x.y;
          }
        }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        // bytes of four keys of one dim in a word, for the two groups of keys
        uint32_t z[2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t t0 = __byte_perm(w[half][0][j], w[half][1][j], 0x5140),
                         t1 = __byte_perm(w[half][2][j], w[half][3][j], 0x5140),
                         t2 = __byte_perm(w[half][0][j], w[half][1][j], 0x7362),
                         t3 = __byte_perm(w[half][2][j], w[half][3][j], 0x7362);
          z[half][0] = __byte_perm(t0, t1, 0x5410);
          z[half][1] = __byte_perm(t0, t1, 0x7632);
          z[half][2] = __byte_perm(t2, t3, 0x5410);
          z[half][3] = __byte_perm(t2, t3, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t A[4] = {z[0][2 * m], z[0][2 * m + 1], z[1][2 * m], z[1][2 * m + 1]};
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (kk == 0) mma_8bit_first(d[r][2 * j + m], A, b[r][0], b[r][1]);
            else mma_8bit(d[r][2 * j + m], A, b[r][2 * kk], b[r][2 * kk + 1]);
          }
        }
      }
      if (2 * kk + 2 == S / 32) half_read();
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        o[r][2 * mt] = C::join(d[r][mt][0], d[r][mt][1]);
        o[r][2 * mt + 1] = C::join(d[r][mt][2], d[r][mt][3]);
      }
  }
};

// ------------------------------------------------------------ half precision ---
template <typename C, int D, int S, int G, int PARTS = 2>
struct HalfOps {
  static constexpr int R = 2;
  static constexpr float kOne = 32768.f, kLog2One = 15.f;
  static HILS_DI int head(int r, int c4) { return 2 * c4 + r; }
  struct Query {
    uint32_t w[PARTS][D / 8];  // nearest half (and rest)
    float up[R];
  };
  static HILS_DI int row_head(int gq) { return gq; }
  template <typename T>
  static HILS_DI void make_query(const RawRow<T, D>& raw, int, int c4, Query& q) {
    float x[D / 4];
    row_values<T, D>(raw, x);
    float largest = 0.f;  // (NaN aside: it stays one in half precision)
#pragma unroll
    for (int i = 0; i < D / 4; ++i) largest = fmaxf(largest, fabsf(x[i]));
    const unsigned top = row_max(__float_as_uint(largest));
    // the power of two that brings the largest element into [2^14, 2^15); 2^14
    // for a row that is zero or not finite
    unsigned ex = top >> 23;
    ex = top == 0 || ex == 255 ? 127 : max(ex, 15u);
    const float down = __uint_as_float((268u - ex) << 23), up = __uint_as_float((ex - 14u) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const float a = x[4 * ks] * down, b = x[4 * ks + C::kX1] * down, c = x[4 * ks + C::kY0] * down,
                  d = x[4 * ks + 3] * down;
      q.w[0][2 * ks] = pack_f16x2(a, b);
      q.w[0][2 * ks + 1] = pack_f16x2(c, d);
      if (PARTS == 2) {
        q.w[PARTS - 1][2 * ks] = rest_f16x2(a, b, q.w[0][2 * ks]);
        q.w[PARTS - 1][2 * ks + 1] = rest_f16x2(c, d, q.w[0][2 * ks + 1]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) q.up[r] = __shfl_sync(0xffffffffu, up, 4 * (2 * c4 + r));
  }
  static HILS_DI void scores(const Tile<D, S>& t, const TileOffsets<D>& at, const Query& q, float (&sc)[R][S / 8]) {
    constexpr int V = D / 64;
#pragma unroll
    for (int mt = 0; mt < S / 16; ++mt) {
      float d[4];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint4 a = *reinterpret_cast<const uint4*>(t.keys16(mt) + at.k[v][0]),
                    b = *reinterpret_cast<const uint4*>(t.keys16(mt) + at.k[v][1]);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t A[4];
          C::halves(wa[j], A[0], A[2]);
          C::halves(wb[j], A[1], A[3]);
          const int ks = 4 * v + j;
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            if (ks == 0 && p == 0) mma_f16_16816_first(d, A, q.w[p][0], q.w[p][1]);
            else mma_f16_16816(d, A, q.w[p][2 * ks], q.w[p][2 * ks + 1]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) sc[r][2 * mt] = d[r], sc[r][2 * mt + 1] = d[2 + r];
    }
  }
  template <typename F>
  static HILS_DI void values(const Tile<D, S>& t, const TileOffsets<D>& at, int, const float (&p)[R][S / 8],
                             float (&o)[R][D / 8], F half_read) {
    constexpr int W = D / 32;  // words of a thread's part of a key
    float d[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < S / 16; ++kk) {
      uint32_t b0[PARTS], b1[PARTS];
      const uint32_t h0 = pack_f16x2(p[0][2 * kk], p[1][2 * kk]), h1 = pack_f16x2(p[0][2 * kk + 1], p[1][2 * kk + 1]);
      b0[0] = movmatrix_trans16(h0);
      b1[0] = movmatrix_trans16(h1);
      if (PARTS == 2) {
        b0[PARTS - 1] = movmatrix_trans16(rest_f16x2(p[0][2 * kk], p[1][2 * kk], h0));
        b1[PARTS - 1] = movmatrix_trans16(rest_f16x2(p[0][2 * kk + 1], p[1][2 * kk + 1], h1));
      }
      uint32_t w[4][W];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* a = t.keys16(kk) + at.v[e];
        if (W == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(a);
          w[e][0] = x.x, w[e][1] = x.y, w[e][W - 2] = x.z, w[e][W - 1] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(a);
          w[e][0] = x.x, w[e][1] = x.y;
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        uint32_t A[4];
        C::halves(C::pair01(w[0][j], w[1][j]), A[0], A[1]);
        C::halves(C::pair01(w[2][j], w[3][j]), A[2], A[3]);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          if (kk == 0 && q == 0) mma_f16_16816_first(d[2 * j], A, b0[q], b1[q]);
          else mma_f16_16816(d[2 * j], A, b0[q], b1[q]);
        }
        C::halves(C::pair23(w[0][j], w[1][j]), A[0], A[1]);
        C::halves(C::pair23(w[2][j], w[3][j]), A[2], A[3]);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          if (kk == 0 && q == 0) mma_f16_16816_first(d[2 * j + 1], A, b0[q], b1[q]);
          else mma_f16_16816(d[2 * j + 1], A, b0[q], b1[q]);
        }
      }
      if (kk + 1 == S / 32) half_read();
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int r = 0; r < R; ++r) o[r][2 * mt] = d[mt][r], o[r][2 * mt + 1] = d[mt][2 + r];
  }
};

}  // namespace hils
