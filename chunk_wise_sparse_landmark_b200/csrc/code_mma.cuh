// Warp-level building blocks for one tile of 8-bit codes (S keys x D dims, one
// byte an element) in shared memory, with up to 8 query columns:
//
//   S^T (S keys x 8 cols)  = X_tile (keys x D) . Q^T (D x cols)
//   O^T (D x 8 cols)       = Y_tile^T (D x keys) . P^T (keys x cols)
//
// half-precision mma.sync m16n8k16 with float32 accumulation.  Every code of
// either format is exact in half precision (int8: integers up to 128; e4m3: 4
// bits of significand, 2^-9 .. 448), so the only roundings are those of Q and P.
// A query row is scaled by the power of two that brings its largest element
// into [1, 2): bf16's 8 bits fit half precision's 11, and what falls below its
// smallest step is off by 2^-25 of the row's largest element.  PARTS = 2 holds
// float32 queries and weights as a sum of two halves (high and rest): off by
// 2^-25 of the largest element as well.
//
// The tile is stored in lines of 128 bytes whose 16-byte pieces are swizzled as
// TMA does (piece i of line r at i ^ (r & 7)); with gq = lane / 4, c4 = lane % 4:
// * S^T: the contraction index is permuted, alike for X and Q: thread c4 holds
//   the D / 4 dims from c4 D / 4 on, whole words of four codes, one word for
//   each k-step.  The eight lanes that share one of a load's phases touch all
//   eight pieces of a line once (no bank conflicts).
// * O^T: row gq of m-tile mt is dim gq D / 8 + 2 mt, row gq + 8 the next one,
//   so a thread's codes of a key are D / 8 contiguous bytes.
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
HILS_DI uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// the rest of (lo, hi) after pack_f16x2
HILS_DI uint32_t rest_f16x2(float lo, float hi, uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_f16x2(lo - f.x, hi - f.y);
}

// ------------------------------------------------------------------- codes ---
// Two halves from two codes.  int8: a byte u = code + 128 below 0x64 is the half
// 1024 + u, so subtracting 1152 leaves the code; even and odd bytes of a word
// are taken apart by one mask.  e4m3: the conversion instruction, by half-words.
struct CodeI8 {
  static constexpr int kFormat = 1;
  // bytes {0, 2} and {1, 3} of w
  static HILS_DI void halves(uint32_t w, uint32_t& x, uint32_t& y) {
    x = sub((w & 0x00ff00ffu) ^ 0x64806480u);
    y = sub(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u);
  }
  static constexpr int kX1 = 2, kY0 = 1;  // x = (byte 0, byte kX1), y = (byte kY0, byte 3)
  // words of two keys -> (a, b) of bytes 0 and 1 (x), of bytes 2 and 3 (y)
  static HILS_DI uint32_t pair01(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
  static HILS_DI uint32_t pair23(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

 private:
  static HILS_DI uint32_t sub(uint32_t h) {
    const uint32_t k = 0x64806480u;  // 1152
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&k));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
struct CodeE4M3 {
  static constexpr int kFormat = 2;
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

// byte offset of linear byte `o` of a tile
HILS_DI int swz(int o) { return o ^ (((o >> 7) & 7) << 4); }

// ------------------------------------------------------------------ queries ---
// Q^T B-fragments of column gq from that column's row (nullptr: zero column),
// and the power of two that the row was divided by.
template <typename T, typename C, int D, int PARTS>
HILS_DI float load_qrow(const T* row, int c4, uint32_t (&qf)[PARTS][D / 8]) {
  constexpr int N = D / 4;  // this thread's dims
  float x[N];
  unsigned top = 0;
  if (row) {
    const uint4* p = reinterpret_cast<const uint4*>(row + c4 * N);
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int v = 0; v < N / PER; ++v) {
      const uint4 w = __ldg(p + v);
      const uint32_t r[4] = {w.x, w.y, w.z, w.w};
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
#pragma unroll
    for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.f;
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // the largest element's exponent (that of 1 for a row that is zero or not finite), less 14
  unsigned ex = top >> 23;
  ex = top == 0 || ex == 255 ? 127 : max(ex, 15u);
  const float down = __uint_as_float((268u - ex) << 23), up = __uint_as_float((ex - 14u) << 23);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const float a = x[4 * ks] * down, b = x[4 * ks + C::kX1] * down, c = x[4 * ks + C::kY0] * down,
                d = x[4 * ks + 3] * down;
    qf[0][2 * ks] = pack_f16x2(a, b);
    qf[0][2 * ks + 1] = pack_f16x2(c, d);
    if (PARTS == 2) {
      qf[PARTS - 1][2 * ks] = rest_f16x2(a, b, qf[0][2 * ks]);
      qf[PARTS - 1][2 * ks + 1] = rest_f16x2(c, d, qf[0][2 * ks + 1]);
    }
  }
  return up;
}

// ------------------------------------------------------------------ products ---
// sc = S^T of the tile: sc[mt][0, 1] key 16 mt + gq, columns 2 c4 and 2 c4 + 1;
// sc[mt][2, 3] key 16 mt + gq + 8
template <typename C, int D, int S, int PARTS>
HILS_DI void tile_scores(const uint8_t* t, int gq, int c4, const uint32_t (&qf)[PARTS][D / 8], float (&sc)[S / 16][4]) {
  constexpr int V = D / 64;  // 16-byte pieces of a thread's row part
#pragma unroll
  for (int mt = 0; mt < S / 16; ++mt) {
    sc[mt][0] = sc[mt][1] = sc[mt][2] = sc[mt][3] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int o = (16 * mt + gq) * D + c4 * (D / 4) + 16 * v;
      const uint4 a = *reinterpret_cast<const uint4*>(t + swz(o));
      const uint4 b = *reinterpret_cast<const uint4*>(t + swz(o + 8 * D));
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t A[4];
        C::halves(wa[j], A[0], A[2]);
        C::halves(wb[j], A[1], A[3]);
        const int ks = 4 * v + j;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) mma_f16_16816(sc[mt], A, qf[p][2 * ks], qf[p][2 * ks + 1]);
      }
    }
  }
}

// o = O^T of the tile with weights p (the layout of sc): o[mt][0, 1] dim
// gq D / 8 + 2 mt of columns 2 c4 and 2 c4 + 1; o[mt][2, 3] the next dim
template <typename C, int D, int S, int PARTS>
HILS_DI void tile_values(const uint8_t* t, int gq, int c4, const float (&p)[S / 16][4], float (&o)[D / 16][4]) {
  constexpr int W = D / 32;  // words of a thread's part of a key
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
#pragma unroll
  for (int kk = 0; kk < S / 16; ++kk) {
    uint32_t b0[PARTS], b1[PARTS];
    const uint32_t h0 = pack_f16x2(p[kk][0], p[kk][1]), h1 = pack_f16x2(p[kk][2], p[kk][3]);
    b0[0] = movmatrix_trans16(h0);
    b1[0] = movmatrix_trans16(h1);
    if (PARTS == 2) {
      b0[PARTS - 1] = movmatrix_trans16(rest_f16x2(p[kk][0], p[kk][1], h0));
      b1[PARTS - 1] = movmatrix_trans16(rest_f16x2(p[kk][2], p[kk][3], h1));
    }
    uint32_t w[4][W];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* a = t + swz((16 * kk + 2 * c4 + (e & 1) + 8 * (e >> 1)) * D + gq * (D / 8));
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
      for (int q = 0; q < PARTS; ++q) mma_f16_16816(o[2 * j], A, b0[q], b1[q]);
      C::halves(C::pair23(w[0][j], w[1][j]), A[0], A[1]);
      C::halves(C::pair23(w[2][j], w[3][j]), A[2], A[3]);
#pragma unroll
      for (int q = 0; q < PARTS; ++q) mma_f16_16816(o[2 * j + 1], A, b0[q], b1[q]);
    }
  }
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
// 2^x (0 for -inf)
HILS_DI float exp2_fast(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
HILS_DI float exp_neg(float x) { return exp2_fast(x * kLog2e); }
// 2^15 e^x, x <= 0
constexpr float kWeight1 = 32768.f;
HILS_DI float weight_of(float x) { return exp2_fast(fmaf(x, kLog2e, 15.f)); }

}  // namespace hils
