// Appending rows to a paged cache with the rotary position embedding applied
// on the way, and reading a cache back.
//
// The hyper.ai summary of arXiv 2607.02980 (HiLS-Attention), section 实验
// (Experiments), counts what a decode step touches; codes of one byte with one
// scale for each chunk and KV head halve it.  A block X (one chunk of one KV
// head, S x d values) with A = max |x| is held as code = rn(x (1 / A * M)), scale
// = A (1 / M), M = 127 (int8) or 448 (e4m3).  It needs the whole block's A, so a
// chunk becomes codes when its last token arrives; its tokens wait in a tail in
// the configuration's type, and what the cache holds does not depend on how
// tokens were split over calls.
//
// One launch with two kinds of CTAs in turn.  One takes a (touched chunk, KV
// head): rows of the call from the projection's output (keys rotated), earlier
// rows of a chunk that completes from the tail, everything in registers between
// load and store.  The other rotates rows of the queries.  Both read each element
// once and write it once.  Alone, the first is bound by its instructions and
// waits (scale, then codes), the second by the memory, so they are mixed: 32768
// rows, 32 heads over 8, int8: 138 us, 5.5 TB/s of the 755 MB it must move (an
// earlier form 141: the kinds one after the other 156, the first kind alone 70 us,
// 2.9 TB/s).  8192 rows into bf16 pages: 35.0 us, 5.9 TB/s; into float32 pages 69.7
// us, 5.8 TB/s.  48 single float32 rows: 3.6 us.
#include <cuda_fp8.h>

#include "launch.h"

namespace hils {
namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 0x1p-110f;

// ------------------------------------------------- eight elements at once ---
// as they are in memory (a thread keeps several of them between load and store)
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
HILS_DI Raw8<T> load_raw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
HILS_DI void store_raw(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
}
HILS_DI void to_values(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.w[i].x), x[4 * i + 1] = __uint_as_float(r.w[i].y);
    x[4 * i + 2] = __uint_as_float(r.w[i].z), x[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
HILS_DI void to_values(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f32x2(w[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
HILS_DI void to_raw(const float (&x)[8], Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
}
HILS_DI void to_raw(const float (&x)[8], Raw8<__nv_bfloat16>& r) {
  r.w[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
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
HILS_DI void rotate_raw(const RopeView& rp, const float (&co)[8], const float (&si)[8], Raw8<T>& r0, Raw8<T>& r1) {
  float x0[8], x1[8];
  to_values(r0, x0);
  to_values(r1, x1);
  rotate(rp, co, si, x0, x1);
  to_raw(x0, r0);
  to_raw(x1, r1);
}

// ------------------------------------------------------------------- codes ---
// Eight codes of x by.  int8: |x by| <= 127 (1 + 2^-21), so adding 1.5 2^23 rounds
// it to an integer of at most 127, in the low byte, to nearest even.
template <int FMT>
HILS_DI uint2 encode8(const float (&x)[8], float by) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(x[4 * h + i], by);
    if (FMT == kI8) {
      uint32_t z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
      w[h] = __byte_perm(__byte_perm(z[0], z[1], 0x0040), __byte_perm(z[2], z[3], 0x0040), 0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3),
                     hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
      w[h] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}
// Largest magnitude of eight elements as the bits of a float32: magnitudes order
// like their bits (NaN above infinity), also those of bf16 pairs in their halves.
HILS_DI unsigned top_bits(unsigned top, const Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    top = max(max(top, max(r.w[i].x & 0x7fffffffu, r.w[i].y & 0x7fffffffu)),
              max(r.w[i].z & 0x7fffffffu, r.w[i].w & 0x7fffffffu));
  return top;
}
HILS_DI unsigned top_bits(unsigned top, const Raw8<__nv_bfloat16>& r) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
  unsigned low = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top = max(top, w[i] & 0x7fff0000u);
    low = max(low, w[i] & 0x00007fffu);
  }
  return max(top, low << 16);
}

// ------------------------------------------------------------- the new rows ---
HILS_DI int row_begin(const NewRows& nr, int b) { return nr.row_start ? __ldg(nr.row_start + b) : b; }
// new rows [r0, r1) of sequence b; false if they do not lie in [0, n_rows) in order
HILS_DI bool seq_rows(const NewRows& nr, int b, int& r0, int& r1) {
  r0 = row_begin(nr, b);
  r1 = row_begin(nr, b + 1);
  return r0 >= 0 && r1 >= r0 && r1 <= nr.n_rows;
}
constexpr int kNobody = 0x7fffffff;
// Whether one of the sequences tid, tid + kThreads .. before b ends behind b's
// first row.  (row_start falls somewhere then; the rows that two sequences name
// are those of the earlier one.)  These loops over sequences are not unrolled: a
// launch fetches its code anew, and a decode step of 16 sequences took 32.8 us for
// 31.8 with them unrolled.
HILS_DI bool begins_inside(const NewRows& nr, int b, int tid) {
  const int first = row_begin(nr, b);
  bool inside = false;
#pragma unroll 1
  for (int x = tid; x < b; x += kThreads) {
    int r0, r1;
    inside = inside || (seq_rows(nr, x, r0, r1) && r1 > first);
  }
  return inside;
}
HILS_DI bool len_fits(const Shape& s, int L, int n) { return L >= 1 && L <= s.N && n <= L; }

// the angle row of new row r at cache position p, or -1 (reported)
HILS_DI int angle_row(const NewRows& nr, const RopeView& rp, int r, int p, const DevCtx& ctx) {
  if (nr.positions) p = __ldg(nr.positions + r);
  if (p >= 0 && p < rp.max_pos) return p;
  raise_status(ctx, kStatusBadIndex);
  return -1;
}


// Block numbers of the two kinds of CTAs, dealt in turn: after each one of the
// fewer kind `per` - 1 of the other, and what is left of those at the end.
struct CtaMix {
  int fewer, per;
  bool fewer_queries;
  HILS_DI int part(int x, bool& queries) const {
    const int round = x / per;
    if (x >= fewer * per) {
      queries = !fewer_queries;
      return x - fewer;
    }
    queries = (x == round * per) == fewer_queries;
    return x == round * per ? round : x - round - 1;
  }
};

template <typename T, int FMT, int D, int S>
__global__ void __launch_bounds__(kThreads, 3) cache_append_kernel(
    Shape s, CacheView cv, DecView dv, NewRows nr, RopeView rp, CtaMix mix, int q_lanes, DevCtx ctx) {
  constexpr int SLOTS = D / 16;  // two groups of eight elements each
  constexpr int STEP = kThreads / SLOTS, NI = (S + STEP - 1) / STEP;  // rows of a pass, passes over a chunk
  constexpr int kHeads = sizeof(T) == 2 ? 4 : 2;  // heads that a thread of the queries' part has in flight
  __shared__ int sh_b, sh_falls;  // whether row_start falls somewhere
  __shared__ int sh_seq[kThreads / 2];
  __shared__ int sh_inside[kThreads / 2];
  __shared__ unsigned sh_top[2][kThreads / 32];
  const unsigned long long zero = grid_begin();
  behind(zero, cv), behind(zero, dv), behind(zero, nr), behind(zero, rp);
  const int tid = threadIdx.x, slot = tid % SLOTS;
  int e0, e1;  // the thread's groups of every row
  slot_groups(slot, rp.rot, e0, e1);
  bool queries;
  const int cta = mix.part(blockIdx.x, queries);

  if (queries) {
    // ---- queries: thread = (row, slot, one of q_lanes heads and those that follow
    // in steps of q_lanes), one load of the angles for all of them.  The first
    // loads are asked for before the row's sequence is known.
    const int per_row = SLOTS * q_lanes, rows = kThreads / per_row;
    const int t0 = cta * rows;
    const int i = tid / per_row, t = t0 + i, h0 = (tid % per_row) / SLOTS;
    const bool live = i < rows && t < nr.n_rows;
    Raw8<T> r0[kHeads], r1[kHeads];
    const T* q = (const T*)nr.q + (long long)t * nr.q_row;
    auto ask = [&](int hb) {
#pragma unroll
      for (int x = 0; x < kHeads; ++x) {
        const int h = hb + x * q_lanes;
        if (live && h < s.Hq) {
          r0[x] = load_raw(q + h * nr.q_head + e0);
          r1[x] = load_raw(q + h * nr.q_head + e1);
        }
      }
    };
    ask(h0);
    if (tid < rows) sh_seq[tid] = kNobody;
    if (tid == 0) sh_falls = 0;
    __syncthreads();
#pragma unroll 1
    for (int b = tid; b < s.B; b += kThreads) {
      int a, z;
      const bool fine = seq_rows(nr, b, a, z);
      if (z < a) sh_falls = 1;
      if (!fine) continue;
#pragma unroll 1
      for (int y = max(a, t0); y < min(z, t0 + rows); ++y) sh_seq[y - t0] = b;
    }
    __syncthreads();
    if (__builtin_expect(sh_falls, 0)) {  // a row may have several: the first of them, if it begins inside no other
      if (tid < rows) sh_inside[tid] = 0;
#pragma unroll 1
      for (int b = tid; b < s.B; b += kThreads) {
        int a, z;
        if (!seq_rows(nr, b, a, z)) continue;
#pragma unroll 1
        for (int y = max(a, t0); y < min(z, t0 + rows); ++y) atomicMin(&sh_seq[y - t0], b);
      }
      __syncthreads();
#pragma unroll 1
      for (int y = 0; y < rows; ++y)
        if (sh_seq[y] != kNobody && begins_inside(nr, sh_seq[y], tid)) sh_inside[y] = 1;
      __syncthreads();
      if (live && sh_inside[i]) return;
    }
    if (!live || sh_seq[i] == kNobody) return;
    const int b = sh_seq[i], a = row_begin(nr, b), z = row_begin(nr, b + 1);
    const int L = dv_len(dv, s, b);
    if (!len_fits(s, L, z - a)) return;  // reported by the cache's part
    int at = -1;
    float co[8], si[8];
    if (16 * slot < rp.rot) {
      at = angle_row(nr, rp, t, L - (z - t), ctx);
      if (at >= 0) load_angles(rp, at, e0, e1, co, si);
    }
    T* o = (T*)nr.q_out + (long long)t * nr.q_out_row;
    for (int hb = h0;;) {
#pragma unroll
      for (int x = 0; x < kHeads; ++x) {
        const int h = hb + x * q_lanes;
        if (h >= s.Hq) break;
        if (at >= 0) rotate_raw(rp, co, si, r0[x], r1[x]);
        store_raw(o + h * nr.q_out_head + e0, r0[x]);
        store_raw(o + h * nr.q_out_head + e1, r1[x]);
      }
      hb += kHeads * q_lanes;
      if (hb >= s.Hq) break;
      ask(hb);
    }
    return;
  }

  // ---- cache: (unit, KV head), keys and values.  Sequence b owns the units from
  // row_start[b] / S + 2 b on: floor(n / S) + 2 of them at least, and n rows
  // touch no more chunks than that.  (Sequences that share units share rows.)
  const int g = cta % s.Hkv, u = cta / s.Hkv;
  int b = -1;
  if (!nr.row_start) {
    b = u / 2;  // one row each: units 2 b and 2 b + 1 (S > 1 rows to a unit of rows)
    if (b >= s.B || u >= (b + 1) / S + 2 * b + 2 || u < b / S + 2 * b) b = -1;
  }
  if (b < 0) {
    if (tid == 0) sh_b = kNobody, sh_falls = 0;
    __syncthreads();
#pragma unroll 1
    for (int x = tid; x < s.B; x += kThreads) {
      int r0, r1;
      const bool fine = seq_rows(nr, x, r0, r1);
      if (r1 < r0) sh_falls = 1;
      if (!fine) {
        if (cta == 0) raise_status(ctx, kStatusBadIndex);
        continue;
      }
      if (u >= r0 / S + 2 * x && u < r1 / S + 2 * x + 2) sh_b = x;
    }
    __syncthreads();
    if (__builtin_expect(sh_falls, 0)) {  // the unit may be several sequences': the first one's, if it begins inside no other
#pragma unroll 1
      for (int x = tid; x < s.B; x += kThreads) {
        int r0, r1;
        if (seq_rows(nr, x, r0, r1) && u >= r0 / S + 2 * x && u < r1 / S + 2 * x + 2) atomicMin(&sh_b, x);
      }
      __syncthreads();
      if (sh_b == kNobody || __syncthreads_or(begins_inside(nr, sh_b, tid))) return;
    }
    b = sh_b;
    if (b == kNobody) return;
  }
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
  long long off = -1;
  if (FMT == kNative || whole) {
    off = dv_chunk(dv, s, b, g, c);
    if (off < 0 && tid == 0) raise_status(ctx, kStatusBadIndex);  // a page outside the pool: never written
  }
  // Rows before `first` of chunk c0, if it completes, are read from its tail slot
  // here while chunks last - 1 and last write their slots: if one of those is the
  // same slot, this CTA writes it, after its reads.
  const bool reads_tail = FMT != kNative && first > c0 * S && c0 < last + ((last + 1) * S <= L);
  const bool later = c > c0 && reads_tail && ((c ^ c0) & 1) == 0;
  if (FMT == kNative ? off < 0 : later && !whole) return;
  const T* src[2] = {(const T*)nr.k + g * nr.k_head, (const T*)nr.v + g * nr.v_head};
  const long long src_row[2] = {nr.k_row, nr.v_row};
  T* tails[2] = {(T*)cv.k_tail, (T*)cv.v_tail};
  void* pools[2] = {cv.k_pool, cv.v_pool};
  float* scales[2] = {cv.k_scale, cv.v_scale};

  // the thread's groups of the new row at position p, and the rotation of a key's
  auto load_new = [&](int x, int p, Raw8<T>& y0, Raw8<T>& y1) {
    const T* row = src[x] + (r0 + p - first) * src_row[x];
    y0 = load_raw(row + e0);
    y1 = load_raw(row + e1);
  };
  auto rotate_new = [&](int p, Raw8<T>& y0, Raw8<T>& y1) {
    if (16 * slot >= rp.rot) return;
    const int at = angle_row(nr, rp, r0 + p - first, p, ctx);
    if (at < 0) return;
    float co[8], si[8];
    load_angles(rp, at, e0, e1, co, si);
    rotate_raw(rp, co, si, y0, y1);
  };
  // of the chunk's row j: the new row, or for a chunk that completes the tail's
  auto load_item = [&](int x, int j, Raw8<T>& y0, Raw8<T>& y1) {
    const int p = c * S + j;
    if (j >= S || p >= L) return;
    if (p >= first) {
      load_new(x, p, y0, y1);
    } else if (FMT != kNative && whole) {
      const T* t = tails[x] + tail_off(s, b, g, c) + j * D;
      y0 = load_raw(t + e0);
      y1 = load_raw(t + e1);
    }
  };
  const int j0 = tid / SLOTS;

  // bf16: keys and values are asked for together, 32 KB of loads in flight for a CTA
  constexpr bool kBoth = sizeof(T) == 2;
  Raw8<T> x0[kBoth ? 2 : 1][NI], x1[kBoth ? 2 : 1][NI];
  if (kBoth) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < NI; ++i) load_item(x, j0 + i * STEP, x0[kBoth ? x : 0][i], x1[kBoth ? x : 0][i]);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    Raw8<T>(&y0)[NI] = x0[kBoth ? x : 0];
    Raw8<T>(&y1)[NI] = x1[kBoth ? x : 0];
    if (!kBoth) {
#pragma unroll
      for (int i = 0; i < NI; ++i) load_item(x, j0 + i * STEP, y0[i], y1[i]);
    }
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int j = j0 + i * STEP, p = c * S + j;
      if (j < S && p >= first && p < L) {
        if (x == 0) rotate_new(p, y0[i], y1[i]);
        if (FMT == kNative) {
          T* page = (T*)pools[x] + off;
          store_raw(page + j * D + e0, y0[i]);
          store_raw(page + j * D + e1, y1[i]);
        } else if (c >= last - 1 && !later) {
          T* t = tails[x] + tail_off(s, b, g, c) + j * D;
          store_raw(t + e0, y0[i]);
          store_raw(t + e1, y1[i]);
        }
      }
      if (FMT != kNative && whole && j < S) {
        top = top_bits(top, y0[i]);
        top = top_bits(top, y1[i]);
      }
    }
    if (FMT == kNative || !whole) continue;
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) sh_top[x][tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, sh_top[x][w]);
    if (off < 0) continue;
    const float A = __uint_as_float(top), M = max_code(FMT);
    const bool fine = top < 0x7f800000u, zero = fine && A < kTiny, held = fine && !zero;
    const float by = held ? __fmul_rn(__frcp_rn(A), M) : 0.f;
    uint8_t* page = (uint8_t*)pools[x] + off;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int j = j0 + i * STEP;
      if (j >= S) continue;
      float z0[8], z1[8];
      to_values(y0[i], z0);
      to_values(y1[i], z1);
      const uint2 none = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(page + j * D + e0) = held ? encode8<FMT>(z0, by) : none;
      *reinterpret_cast<uint2*>(page + j * D + e1) = held ? encode8<FMT>(z1, by) : none;
    }
    if (tid == 0)
      scales[x][off / (S * D)] = !fine ? __uint_as_float(0x7fc00000u) : zero ? 0.f : __fmul_rn(A, 1.f / M);
  }
  if (FMT != kNative && whole && c == c0 && reads_tail) {  // every thread has read its tail rows (the barriers above)
    for (int cc = max(last - 1, c0 + 1); cc <= last; ++cc) {
      if ((cc ^ c0) & 1) continue;
      for (int j = j0; j < S && cc * S + j < L; j += STEP) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Raw8<T> y0, y1;
          load_new(x, cc * S + j, y0, y1);
          if (x == 0) rotate_new(cc * S + j, y0, y1);
          T* t = tails[x] + tail_off(s, b, g, cc) + j * D;
          store_raw(t + e0, y0);
          store_raw(t + e1, y1);
        }
      }
    }
  }
}

template <typename T, int FMT, int D, int S>
cudaError_t go_append(const Shape& s, const CacheView& cv, const DecView& dv, const NewRows& nr, const RopeView& rp,
                      cudaStream_t st, const DevCtx& ctx) {
  constexpr int SLOTS = D / 16;
  const long long kv = ((long long)nr.n_rows / S + 2ll * s.B) * s.Hkv;
  // lanes of a row: all heads at once for few rows (latency); a quarter (float32:
  // half) of them for many, so that one load of the angles serves several heads.
  // 32 heads over 8, us, all : part.  bf16 pages, d = 128: 16 rows 3.2 : 3.3, 256
  // 5.0 : 4.6, 1024 9.1 : 7.0, 2048 14.9 : 11.0, 16384 103 : 70.  float32, d = 64:
  // 256 4.9 : 5.4, 1024 8.1 : 9.1, 2048 13.0 : 13.4, 4096 23.6 : 23.7, 16384 90 : 80.
  // So 2048 is float32's border; from 64 to 2047 bf16 rows part would be shorter.
  constexpr int per = sizeof(T) == 2 ? 4 : 2;
  int lanes = s.Hq < kThreads / SLOTS ? s.Hq : kThreads / SLOTS;
  if (nr.n_rows >= 2048) lanes = (lanes + per - 1) / per;
  int rows = kThreads / (SLOTS * lanes);
  if (rows > kThreads / 2) rows = kThreads / 2;
  const long long qc = nr.q ? (nr.n_rows + rows - 1) / rows : 0;
  if (kv + qc > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const long long few = kv < qc ? kv : qc, many = kv < qc ? qc : kv;
  CtaMix mix;
  mix.fewer = (int)few;
  mix.per = few ? (int)(many / few) + 1 : 1;
  mix.fewer_queries = qc <= kv;
  return launch_overlapped(cache_append_kernel<T, FMT, D, S>, dim3((unsigned)(kv + qc)), kThreads, 0, 1, st, s, cv, dv,
                           nr, rp, mix, lanes, ctx);
}

// ------------------------------------------------------------- reading back ---
HILS_DI float decode1(int8_t c) { return (float)c; }
HILS_DI float decode1(__nv_fp8_e4m3 c) { return (float)c; }

// 32 bytes: a whole sector at once where the output is aligned to it
HILS_DI void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
HILS_DI void store16(float* p, const float (&x)[16], bool wide) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[8 * h + i]);
    store32(p + 8 * h, w, wide);
  }
}
HILS_DI void store16(__nv_bfloat16* p, const float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  store32(p, w, wide);
}

// One CTA per (chunk, KV head, sequence; keys or values): a tile is contiguous
// in the pool and in the output.  Bound by memory: 32768 rows, 8 heads, int8 to
// bf16: 34.0 us, 5.9 TB/s.
template <typename T, typename C>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(Shape s, CacheView cv, DecView dv, T* __restrict__ k_out,
                                                              T* __restrict__ v_out, int out_rows, DevCtx ctx) {
  constexpr bool coded = sizeof(C) == 1;
  const unsigned long long zero = grid_begin();
  behind(zero, cv), behind(zero, dv);
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
  const bool in_tail = coded && (c + 1) * s.S > L;  // the incomplete chunk
  const long long off = in_tail ? 0 : dv_chunk(dv, s, b, g, c);
  if (off < 0) {
    if (threadIdx.x == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  if (!coded || in_tail) {
    const T* t = in_tail ? (const T*)(vals ? cv.v_tail : cv.k_tail) + tail_off(s, b, g, c)
                         : (const T*)(vals ? cv.v_pool : cv.k_pool) + off;
#pragma unroll 4
    for (int e = threadIdx.x * 8; e < n; e += kThreads * 8) store_raw(out + e, load_raw(t + e));
    return;
  }
  const C* page = (const C*)(vals ? cv.v_pool : cv.k_pool) + off;
  const float scale = __ldg((vals ? cv.v_scale : cv.k_scale) + off / (s.S * s.d));
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
#pragma unroll 2
  for (int e = threadIdx.x * 16; e < n; e += kThreads * 16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(page + e));
    float x[16];
    const C* codes = reinterpret_cast<const C*>(&w);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = decode1(codes[i]) * scale;
    store16(out + e, x, wide);
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
#define HILS_GO(T, C) \
  return launch_overlapped(cache_read_kernel<T, C>, grid, kThreads, 0, 1, st, s, cv, dv, (T*)k_out, (T*)v_out, out_rows, ctx)
  if (s.dtype == 0) {
    if (cv.format == kI8) HILS_GO(float, int8_t);
    if (cv.format == kE4M3) HILS_GO(float, __nv_fp8_e4m3);
    HILS_GO(float, float);
  }
  if (cv.format == kI8) HILS_GO(__nv_bfloat16, int8_t);
  if (cv.format == kE4M3) HILS_GO(__nv_bfloat16, __nv_fp8_e4m3);
  HILS_GO(__nv_bfloat16, __nv_bfloat16);
#undef HILS_GO
}

}  // namespace hils
