// Appending rows to a paged cache with the rotary position embedding applied
// on the way, and reading a cache back.
//
// The hyper.ai summary of arXiv 2607.02980 (HiLS-Attention), section 实验
// (Experiments), counts what a decode step touches; codes of one byte with one
// scale for each chunk and KV head halve it.  A block X (one chunk of one KV
// head, S x d values) with A = max |x| is held as code = rn(x (M / A)), scale =
// A / M, M = 127 (int8) or 448 (e4m3).  It needs the whole block's A, so a
// chunk becomes codes when its last token arrives; its tokens wait in a tail in
// the configuration's type, and what the cache holds does not depend on how
// tokens were split over calls.
//
// One launch.  The first CTAs take one (touched chunk, KV head, key or value)
// each: rows of the call from the projection's output (keys rotated), earlier
// rows of a chunk that completes from the tail, everything in registers
// between load and store.  The others rotate the queries.
// Both parts read each element once and write it once: memory-bound for
// prompts, latency-bound (three dependent loads) for single tokens.
#include <cuda_fp8.h>

#include "launch.h"

namespace hils {
namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 0x1p-110f;

// ------------------------------------------------- eight elements at once ---
HILS_DI void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
HILS_DI void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f32x2(r[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
HILS_DI void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
HILS_DI void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// ---------------------------------------------------------------- rotation ---
// A thread's slot: two groups of eight elements, e0 and e1.  The first rot / 16
// slots hold both elements of eight pairs (x[i], x[i + rot / 2]); for
// interleaved pairs the same groups hold four whole pairs each.  The rest of
// the row is not rotated.
HILS_DI void slot_groups(int slot, int rot, int& e0, int& e1) {
  if (16 * slot < rot) {
    e0 = 8 * slot;
    e1 = e0 + rot / 2;
  } else {
    e0 = 16 * slot;
    e1 = e0 + 8;
  }
}
HILS_DI void angles4(const float* t, float (&x)[8], int at) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(t));
  x[at] = a.x, x[at + 1] = a.y, x[at + 2] = a.z, x[at + 3] = a.w;
}
// cos and sin of the slot's pairs: halves: pairs 8 slot ..; interleaved: pairs
// e0 / 2 .. + 3, then e1 / 2 .. + 3
HILS_DI void load_angles(const RopeView& rp, int row, int e0, int e1, float (&co)[8], float (&si)[8]) {
  const long long base = (long long)row * (rp.rot / 2);
  const int p0 = rp.interleaved ? e0 / 2 : e0, p1 = rp.interleaved ? e1 / 2 : e0 + 4;
  angles4(rp.cos_t + base + p0, co, 0);
  angles4(rp.cos_t + base + p1, co, 4);
  angles4(rp.sin_t + base + p0, si, 0);
  angles4(rp.sin_t + base + p1, si, 4);
}
// (a, c) -> (a cos - c sin, c cos + a sin); the products are rounded apart (no
// fused multiply-add), so that the result does not depend on the compiler
HILS_DI void turn(float& a, float& c, float co, float si) {
  const float ra = __fsub_rn(__fmul_rn(a, co), __fmul_rn(c, si));
  const float rc = __fadd_rn(__fmul_rn(c, co), __fmul_rn(a, si));
  a = ra, c = rc;
}
HILS_DI void rotate(const RopeView& rp, const float (&co)[8], const float (&si)[8], float (&x0)[8], float (&x1)[8]) {
  if (rp.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(x0[2 * i], x0[2 * i + 1], co[i], si[i]);
      turn(x1[2 * i], x1[2 * i + 1], co[4 + i], si[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x0[i], x1[i], co[i], si[i]);
  }
}
template <typename T>
HILS_DI void round8(float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f32(from_f32<T>(x[i]));
}

// ------------------------------------------------------------------- codes ---
template <int FMT>
HILS_DI uint2 encode8(const float (&x)[8], float by) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __fmul_rn(x[2 * i], by), c = __fmul_rn(x[2 * i + 1], by);
    uint32_t two;
    if (FMT == kI8) {
      const int ia = max(-127, min(127, __float2int_rn(a))), ic = max(-127, min(127, __float2int_rn(c)));
      two = (uint32_t)(ia & 0xff) | ((uint32_t)(ic & 0xff) << 8);
    } else {
      two = __nv_cvt_float2_to_fp8x2(make_float2(a, c), __NV_SATFINITE, __NV_E4M3);
    }
    w[i >> 1] |= two << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}

// ------------------------------------------------------------- the new rows ---
HILS_DI int row_begin(const NewRows& nr, int b) { return nr.row_start ? __ldg(nr.row_start + b) : b; }
// new rows [r0, r1) of sequence b; false if they do not lie in [0, n_rows) in order
HILS_DI bool seq_rows(const NewRows& nr, int b, int& r0, int& r1) {
  r0 = row_begin(nr, b);
  r1 = row_begin(nr, b + 1);
  return r0 >= 0 && r1 >= r0 && r1 <= nr.n_rows;
}
HILS_DI bool len_fits(const Shape& s, int L, int n) { return L >= 1 && L <= s.N && n <= L; }

// the angle row of new row r at cache position p, or -1 (reported)
HILS_DI int angle_row(const NewRows& nr, const RopeView& rp, int r, int p, const DevCtx& ctx) {
  if (nr.positions) p = __ldg(nr.positions + r);
  if (p >= 0 && p < rp.max_pos) return p;
  raise_status(ctx, kStatusBadIndex);
  return -1;
}

template <typename T, int FMT, int D, int S>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(Shape s, CacheView cv, DecView dv, NewRows nr,
                                                                RopeView rp, int kv_ctas, int q_lanes, DevCtx ctx) {
  constexpr int SLOTS = D / 16;  // two groups of eight elements each
  constexpr int ITEMS = S * SLOTS, NI = (ITEMS + kThreads - 1) / kThreads;
  __shared__ int sh_b;
  __shared__ int sh_seq[kThreads / 2];
  __shared__ unsigned sh_top[kThreads / 32];
  const int tid = threadIdx.x;

  if ((int)blockIdx.x >= kv_ctas) {
    // ---- queries: thread = (row, slot, one of q_lanes heads), heads in strides,
    // so that a row's angles are loaded once for several heads
    if (!nr.q) return;
    const int per_row = SLOTS * q_lanes, rows = kThreads / per_row;
    const int t0 = ((int)blockIdx.x - kv_ctas) * rows;
    if (tid < rows) sh_seq[tid] = -1;
    __syncthreads();
    for (int b = tid; b < s.B; b += kThreads) {
      int r0, r1;
      if (!seq_rows(nr, b, r0, r1)) continue;
      for (int t = max(r0, t0); t < min(r1, t0 + rows); ++t) sh_seq[t - t0] = b;
    }
    __syncthreads();
    const int i = tid / per_row;
    if (i >= rows || sh_seq[i] < 0) return;
    const int b = sh_seq[i], t = t0 + i;
    const int r0 = row_begin(nr, b), r1 = row_begin(nr, b + 1);
    const int L = dv_len(dv, s, b);
    if (!len_fits(s, L, r1 - r0)) return;  // reported by the cache's part
    const int slot = tid % SLOTS;
    int e0, e1;
    slot_groups(slot, rp.rot, e0, e1);
    int at = -1;
    float co[8], si[8];
    if (16 * slot < rp.rot) {
      at = angle_row(nr, rp, t, L - (r1 - t), ctx);
      if (at >= 0) load_angles(rp, at, e0, e1, co, si);
    }
    const T* q = (const T*)nr.q + (long long)t * nr.q_row;
    T* o = (T*)nr.q_out + (long long)t * nr.q_out_row;
    for (int h = (tid % per_row) / SLOTS; h < s.Hq; h += q_lanes) {
      float x0[8], x1[8];
      load8(q + h * nr.q_head + e0, x0);
      load8(q + h * nr.q_head + e1, x1);
      if (at >= 0) rotate(rp, co, si, x0, x1);
      store8(o + h * nr.q_out_head + e0, x0);
      store8(o + h * nr.q_out_head + e1, x1);
    }
    return;
  }

  // ---- cache: (unit, KV head, key or value).  Sequence b owns the units from
  // row_start[b] / S + 2 b on: floor(n / S) + 2 of them at least, and n rows
  // touch no more chunks than that.
  const int vals = blockIdx.x & 1, g = (int)(blockIdx.x >> 1) % s.Hkv, u = (int)(blockIdx.x >> 1) / s.Hkv;
  if (tid == 0) sh_b = -1;
  __syncthreads();
  for (int b = tid; b < s.B; b += kThreads) {
    int r0, r1;
    if (!seq_rows(nr, b, r0, r1)) {
      if (blockIdx.x == 0) raise_status(ctx, kStatusBadIndex);
      continue;
    }
    if (u >= r0 / S + 2 * b && u < r1 / S + 2 * b + 2) sh_b = b;
  }
  __syncthreads();
  const int b = sh_b;
  if (b < 0) return;
  const int r0 = row_begin(nr, b), n = row_begin(nr, b + 1) - r0;
  if (n == 0) return;
  const int L = dv_len(dv, s, b);
  if (!len_fits(s, L, n)) {
    if (tid == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  const int first = L - n, c0 = first / S, last = (L - 1) / S;
  const int c = c0 + (u - r0 / S - 2 * b);
  if (c > last) return;
  const bool whole = (c + 1) * S <= L;
  const bool rot = !vals && rp.rot > 0;
  const T* src = (const T*)(vals ? nr.v : nr.k) + g * (vals ? nr.v_head : nr.k_head);
  const long long src_row = vals ? nr.v_row : nr.k_row;
  long long off = -1;
  if (FMT == kNative || whole) {
    off = dv_chunk(dv, s, b, g, c);
    if (off < 0 && tid == 0) raise_status(ctx, kStatusBadIndex);  // a page outside the pool: never written
  }
  T* tail = FMT == kNative ? nullptr : (T*)(vals ? cv.v_tail : cv.k_tail);

  // new row of chunk cc at j, its slot's two groups, rotated and rounded to T
  auto load_new = [&](int cc, int j, int slot, int e0, int e1, float (&x0)[8], float (&x1)[8]) {
    const int p = cc * S + j, r = r0 + p - first;
    load8(src + r * src_row + e0, x0);
    load8(src + r * src_row + e1, x1);
    if (rot && 16 * slot < rp.rot) {
      const int at = angle_row(nr, rp, r, p, ctx);
      if (at >= 0) {
        float co[8], si[8];
        load_angles(rp, at, e0, e1, co, si);
        rotate(rp, co, si, x0, x1);
        round8<T>(x0);
        round8<T>(x1);
      }
    }
  };

  if constexpr (FMT == kNative) {
    if (off < 0) return;
    T* page = (T*)(vals ? cv.v_pool : cv.k_pool) + off;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int item = tid + i * kThreads, j = item / SLOTS, slot = item % SLOTS;
      if (item >= ITEMS || c * S + j < first || c * S + j >= L) continue;
      int e0, e1;
      slot_groups(slot, rp.rot, e0, e1);
      float x0[8], x1[8];
      load_new(c, j, slot, e0, e1, x0, x1);
      store8(page + j * D + e0, x0);
      store8(page + j * D + e1, x1);
    }
  } else {
    // Rows before `first` of chunk c0, if it completes, are read from its tail
    // slot here while chunks last - 1 and last write their slots: if one of
    // those is the same slot, this CTA writes it, after its reads.
    const bool reads_tail = first > c0 * S && c0 < last + ((last + 1) * S <= L);
    const bool later = c > c0 && reads_tail && ((c ^ c0) & 1) == 0;
    if (later && !whole) return;
    float x0[NI][8], x1[NI][8];
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int item = tid + i * kThreads, j = item / SLOTS, slot = item % SLOTS, p = c * S + j;
      const bool is_new = item < ITEMS && p >= first && p < L;
      if (!is_new && !(whole && item < ITEMS)) continue;
      int e0, e1;
      slot_groups(slot, rp.rot, e0, e1);
      if (is_new) {
        load_new(c, j, slot, e0, e1, x0[i], x1[i]);
        if (c >= last - 1 && !later) {
          T* t = tail + tail_off(s, b, g, c) + j * D;
          store8(t + e0, x0[i]);
          store8(t + e1, x1[i]);
        }
      } else {
        const T* t = tail + tail_off(s, b, g, c) + j * D;
        load8(t + e0, x0[i]);
        load8(t + e1, x1[i]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)  // magnitudes order like their bits; NaN above infinity
        top = max(top, max(__float_as_uint(x0[i][k]) & 0x7fffffffu, __float_as_uint(x1[i][k]) & 0x7fffffffu));
    }
    if (!whole) return;
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) sh_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, sh_top[w]);
    if (off >= 0) {
      const float A = __uint_as_float(top), M = max_code(FMT);
      const bool fine = top < 0x7f800000u, zero = fine && A < kTiny, held = fine && !zero;
      const float by = held ? __fdiv_rn(M, A) : 0.f;
      uint8_t* page = (uint8_t*)(vals ? cv.v_pool : cv.k_pool) + off;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int item = tid + i * kThreads, j = item / SLOTS, slot = item % SLOTS;
        if (item >= ITEMS) continue;
        int e0, e1;
        slot_groups(slot, rp.rot, e0, e1);
        const uint2 z = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(page + j * D + e0) = held ? encode8<FMT>(x0[i], by) : z;
        *reinterpret_cast<uint2*>(page + j * D + e1) = held ? encode8<FMT>(x1[i], by) : z;
      }
      if (tid == 0)
        (vals ? cv.v_scale : cv.k_scale)[off / (S * D)] =
            !fine ? __uint_as_float(0x7fc00000u) : zero ? 0.f : __fdiv_rn(A, M);
    }
    if (c == c0 && reads_tail) {
      for (int cc = max(last - 1, c0 + 1); cc <= last; ++cc) {
        if ((cc ^ c0) & 1) continue;
        for (int item = tid; item < ITEMS; item += kThreads) {
          const int j = item / SLOTS, slot = item % SLOTS;
          if (cc * S + j >= L) continue;
          int e0, e1;
          slot_groups(slot, rp.rot, e0, e1);
          float y0[8], y1[8];
          load_new(cc, j, slot, e0, e1, y0, y1);
          T* t = tail + tail_off(s, b, g, cc) + j * D;
          store8(t + e0, y0);
          store8(t + e1, y1);
        }
      }
    }
  }
}

template <typename T, int FMT, int D, int S>
cudaError_t go_append(const Shape& s, const CacheView& cv, const DecView& dv, const NewRows& nr, const RopeView& rp,
                      cudaStream_t st, const DevCtx& ctx) {
  constexpr int SLOTS = D / 16;
  const long long kv = ((long long)nr.n_rows / S + 2ll * s.B) * s.Hkv * 2;
  // lanes of a row: all heads for few rows (latency); a quarter of them for
  // many, so that one load of the angles serves four heads
  int lanes = s.Hq < kThreads / SLOTS ? s.Hq : kThreads / SLOTS;
  if (nr.n_rows >= 2048 && lanes >= 4) lanes /= 4;
  int rows = kThreads / (SLOTS * lanes);
  if (rows > kThreads / 2) rows = kThreads / 2;
  const long long qc = nr.q ? (nr.n_rows + rows - 1) / rows : 0;
  if (kv + qc > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cache_append_kernel<T, FMT, D, S>
      <<<(unsigned)(kv + qc), kThreads, 0, st>>>(s, cv, dv, nr, rp, (int)kv, lanes, ctx);
  return cudaGetLastError();
}

// ------------------------------------------------------------- reading back ---
HILS_DI float decode1(int8_t c) { return (float)c; }
HILS_DI float decode1(__nv_fp8_e4m3 c) { return (float)c; }
HILS_DI float decode1(float c) { return c; }
HILS_DI float decode1(__nv_bfloat16 c) { return to_f32(c); }

// One CTA per (chunk, KV head, sequence; keys or values): a tile is contiguous
// in the pool and in the output.  Thread: groups of eight elements.
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(Shape s, CacheView cv, DecView dv, T* __restrict__ k_out,
                                                              T* __restrict__ v_out, int out_rows, DevCtx ctx) {
  constexpr bool coded = sizeof(C) == 1;
  const int c = blockIdx.x, g = blockIdx.y >> 1, b = blockIdx.z, vals = blockIdx.y & 1;
  T* out = vals ? v_out : k_out;
  if (!out) return;
  const int L = dv_len(dv, s, b);
  if (L < 0 || L > s.N) {
    if (threadIdx.x == 0 && c == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  const int rows = min(min(s.S, L - c * s.S), out_rows - c * s.S);
  if (rows <= 0) return;
  out += (((long long)b * s.Hkv + g) * out_rows + (long long)c * s.S) * s.d;
  const int n = rows * s.d;
  if (coded && (c + 1) * s.S > L) {  // the incomplete chunk
    const T* t = (const T*)(vals ? cv.v_tail : cv.k_tail) + tail_off(s, b, g, c);
    for (int e = threadIdx.x * 8; e < n; e += kThreads * 8) {
      float x[8];
      load8(t + e, x);
      store8(out + e, x);
    }
    return;
  }
  const long long off = dv_chunk(dv, s, b, g, c);
  if (off < 0) {
    if (threadIdx.x == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  const C* page = (const C*)(vals ? cv.v_pool : cv.k_pool) + off;
  if constexpr (coded) {
    const float scale = __ldg((vals ? cv.v_scale : cv.k_scale) + off / (s.S * s.d));
    for (int e = threadIdx.x * 8; e < n; e += kThreads * 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(page + e);
      float x[8];
      const C* codes = reinterpret_cast<const C*>(&w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = decode1(codes[i]) * scale;
      store8(out + e, x);
    }
  } else {
    for (int e = threadIdx.x * 8; e < n; e += kThreads * 8) {
      float x[8];
      load8(page + e, x);
      store8(out + e, x);
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const Shape& s, const CacheView& cv, const DecView& dv, const NewRows& nr,
                                const RopeView& rp, cudaStream_t st, const DevCtx& ctx) {
#define HILS_CASE(T, F, DD, SS) \
  if (cv.format == F && s.d == DD && s.S == SS) return go_append<T, F, DD, SS>(s, cv, dv, nr, rp, st, ctx);
  if (s.dtype == 0) {
    HILS_CASE(float, kNative, 32, 16) HILS_CASE(float, kNative, 32, 32)
    HILS_CASE(float, kNative, 64, 16) HILS_CASE(float, kNative, 64, 32) HILS_CASE(float, kNative, 64, 64)
    HILS_CASE(float, kNative, 128, 16) HILS_CASE(float, kNative, 128, 32) HILS_CASE(float, kNative, 128, 64)
    HILS_CASE(float, kI8, 64, 32) HILS_CASE(float, kI8, 64, 64)
    HILS_CASE(float, kI8, 128, 32) HILS_CASE(float, kI8, 128, 64)
    HILS_CASE(float, kE4M3, 64, 32) HILS_CASE(float, kE4M3, 64, 64)
    HILS_CASE(float, kE4M3, 128, 32) HILS_CASE(float, kE4M3, 128, 64)
  } else {
    HILS_CASE(__nv_bfloat16, kNative, 128, 64)
    HILS_CASE(__nv_bfloat16, kI8, 128, 64)
    HILS_CASE(__nv_bfloat16, kE4M3, 128, 64)
  }
#undef HILS_CASE
  return cudaErrorNotSupported;
}

cudaError_t launch_cache_read(const Shape& s, const CacheView& cv, const DecView& dv, void* k_out, void* v_out,
                              int out_rows, cudaStream_t st, const DevCtx& ctx) {
  const int chunks = ((out_rows < s.N ? out_rows : s.N) + s.S - 1) / s.S;
  const dim3 grid(chunks, 2 * s.Hkv, s.B);
#define HILS_GO(T, C) cache_read_kernel<T, C><<<grid, kThreads, 0, st>>>(s, cv, dv, (T*)k_out, (T*)v_out, out_rows, ctx)
  if (s.dtype == 0) {
    if (cv.format == kI8) HILS_GO(float, int8_t);
    else if (cv.format == kE4M3) HILS_GO(float, __nv_fp8_e4m3);
    else HILS_GO(float, float);
  } else {
    if (cv.format == kI8) HILS_GO(__nv_bfloat16, int8_t);
    else if (cv.format == kE4M3) HILS_GO(__nv_bfloat16, __nv_fp8_e4m3);
    else HILS_GO(__nv_bfloat16, __nv_bfloat16);
  }
#undef HILS_GO
  return cudaGetLastError();
}

}  // namespace hils
