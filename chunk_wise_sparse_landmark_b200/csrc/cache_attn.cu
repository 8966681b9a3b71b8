// Landmark summaries and decode attention over a paged cache of 8-bit codes
// (cache_append.cu: value = code * scale, one scale for each chunk and KV
// head; a sequence's incomplete chunk in its tail), and summaries over a
// native cache.
//
// hyper.ai summary of arXiv 2607.02980 (HiLS-Attention), section 方法 (Method):
// the summaries k'_c = sum_j p_j k_j, b'_c = H(p), p = softmax_j(q'_c.k_j scale),
// and the token weights w_{i,j} = exp(s_ij) / Z_{i,c} * exp(s^_{i,c}) / Z^_i.
// With k_j = a x_j (a the block's scale, x_j codes) the logit is (q.x_j) a scale
// and the block's output (sum_j p_j y_j) a_v: a scale is applied once for a
// logit and once for an output element, never to a code.
#include <cuda_fp8.h>

#include "launch.h"

namespace hils {
namespace {

constexpr int kThreads = 256;

template <typename C> HILS_DI float code_f32(C c) { return (float)c; }
template <> HILS_DI float code_f32<__nv_bfloat16>(__nv_bfloat16 c) { return __bfloat162float(c); }

// e^{a - M} for a <= M; 0 for a = -inf, also against M = -inf; NaN for a NaN
HILS_DI float rel_weight(float a, float M) { return a == -INFINITY ? 0.f : expf(a - M); }

// a tile of S x D elements of type C into shared memory as float32
template <typename C, int D, int S>
HILS_DI void load_tile(const C* src, int rows, float (&t)[S][D + 1]) {
  for (int e = threadIdx.x; e < S * D; e += kThreads) t[e / D][e % D] = e / D < rows ? code_f32(src[e]) : 0.f;
}

// logits of G queries against the tile's keys, scaled; -inf from row nk on
template <int D, int S, int G>
HILS_DI void tile_logits(const float (&qs)[G][D], const float (&t)[S][D + 1], float scale, int nk, float (&lg)[G][S]) {
  for (int p = threadIdx.x; p < G * S; p += kThreads) {
    const int h = p / S, j = p % S;
    float acc = 0.f;
#pragma unroll 8
    for (int e = 0; e < D; ++e) acc = fmaf(qs[h][e], t[j][e], acc);
    lg[h][j] = j < nk ? acc * scale : -INFINITY;
  }
}

template <typename T, typename C, int D, int S, int G>
__global__ void __launch_bounds__(kThreads) cache_summaries_kernel(Shape s, CacheView cv, DecView dv,
                                                                   const T* __restrict__ q_lmk, LmkStrides ls,
                                                                   const int* __restrict__ from, T* __restrict__ k_sum,
                                                                   float* __restrict__ b_sum, DevCtx ctx) {
  extern __shared__ __align__(16) unsigned char smem[];
  float(&ks)[S][D + 1] = *reinterpret_cast<float(*)[S][D + 1]>(smem);
  __shared__ float qs[G][D];
  __shared__ float lg[G][S];
  const int tid = threadIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = dv_len(dv, s, b), F = from ? __ldg(from + b) : 0;
  if (L < 1 || L > s.N || F < 0) {
    if (tid == 0 && blockIdx.x == 0 && g == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  for (int c = F / S + blockIdx.x; c < L / S; c += gridDim.x) {
    const long long off = dv_chunk(dv, s, b, g, c);
    if (off < 0) {  // a page outside the pool: reported, never read
      if (tid == 0) raise_status(ctx, kStatusBadIndex);
      continue;
    }
    const float scale = sizeof(C) == 1 ? __ldg(cv.k_scale + off / (S * D)) : 1.f;
    load_tile<C, D, S>((const C*)cv.k_pool + off, S, ks);
    for (int e = tid; e < G * D; e += kThreads) qs[e / D][e % D] = to_f32(q_lmk[ls.of(b, g * G + e / D, c) + e % D]);
    __syncthreads();
    tile_logits<D, S, G>(qs, ks, s.scale * scale, S, lg);
    __syncthreads();
    const int warp = tid >> 5, lane = tid & 31;
    for (int h = warp; h < G; h += kThreads / 32) {
      float m = -INFINITY;
      for (int j = lane; j < S; j += 32) m = fmaxf(m, lg[h][j]);
      m = warp_max(m);
      float z = 0.f, zl = 0.f;
      for (int j = lane; j < S; j += 32) {
        const float l = lg[h][j] - m, e = expf(l);
        z += e;
        zl += e * l;
      }
      z = warp_sum(z);
      zl = warp_sum(zl);
      for (int j = lane; j < S; j += 32) lg[h][j] = expf(lg[h][j] - m) / z;
      if (lane == 0) b_sum[((long long)b * s.Hq + g * G + h) * s.C + c] = logf(z) - zl / z;
    }
    __syncthreads();
    for (int o = tid; o < G * D; o += kThreads) {
      const int h = o / D, e = o % D;
      float acc = 0.f;
#pragma unroll 8
      for (int j = 0; j < S; ++j) acc = fmaf(lg[h][j], ks[j][e], acc);
      k_sum[(((long long)b * s.Hq + g * G + h) * s.C + c) * D + e] = from_f32<T>(acc * scale);
    }
    __syncthreads();
  }
}

template <typename T, typename C, int D, int S, int G>
__global__ void __launch_bounds__(kThreads) attn_codes_kernel(Shape s, const T* __restrict__ q, CacheView cv,
                                                              DecView dv, const int32_t* __restrict__ idx,
                                                              const float* __restrict__ s_sel, T* __restrict__ out,
                                                              DevCtx ctx) {
  extern __shared__ __align__(16) unsigned char smem[];
  float(&t)[S][D + 1] = *reinterpret_cast<float(*)[S][D + 1]>(smem);
  __shared__ float qs[G][D];
  __shared__ float lg[G][S];
  __shared__ float sa[G], sz[G];
  const int tid = threadIdx.x, g = blockIdx.x, b = blockIdx.y;
  const int L = dv_len(dv, s, b);
  if (L < 1 || L > s.N) {
    if (tid == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  const int cur = (L - 1) / S, wc0 = max(0, cur - s.nw + 1);
  const int32_t* ir = idx + ((long long)b * s.Hkv + g) * s.K;
  for (int e = tid; e < G * D; e += kThreads) qs[e / D][e % D] = to_f32(q[((long long)b * s.Hq + g * G + e / D) * D + e % D]);
  constexpr int OUTS = (G * D + kThreads - 1) / kThreads;
  float num[OUTS], M[G], den[G];
#pragma unroll
  for (int r = 0; r < OUTS; ++r) num[r] = 0.f;
#pragma unroll
  for (int h = 0; h < G; ++h) M[h] = -INFINITY, den[h] = 0.f;
  for (int u = 0; u < s.K + cur - wc0 + 1; ++u) {
    const bool sel = u < s.K;
    int c = wc0 + u - s.K;
    if (sel) {
      c = ir[u];
      if (!list_entry_accepted(ir, u, wc0)) {  // the list form, common.cuh
        if (c != -1 && tid == 0) raise_status(ctx, kStatusBadIndex);
        continue;
      }
    }
    const int nk = min(S, L - c * S);
    const bool in_tail = nk < S;
    const long long off = in_tail ? tail_off(s, b, g, c) : dv_chunk(dv, s, b, g, c);
    if (off < 0) {  // a page outside the pool: reported, never read
      if (tid == 0) raise_status(ctx, kStatusBadIndex);
      continue;
    }
    const float ks = in_tail ? 1.f : __ldg(cv.k_scale + off / (S * D)), vs = in_tail ? 1.f : __ldg(cv.v_scale + off / (S * D));
    __syncthreads();
    if (in_tail) load_tile<T, D, S>((const T*)cv.k_tail + off, nk, t);
    else load_tile<C, D, S>((const C*)cv.k_pool + off, nk, t);
    __syncthreads();
    tile_logits<D, S, G>(qs, t, s.scale * ks, nk, lg);
    __syncthreads();
    if (in_tail) load_tile<T, D, S>((const T*)cv.v_tail + off, nk, t);
    else load_tile<C, D, S>((const C*)cv.v_pool + off, nk, t);
    const int warp = tid >> 5, lane = tid & 31;
    for (int h = warp; h < G; h += kThreads / 32) {
      float m = -INFINITY;
      for (int j = lane; j < S; j += 32) m = fmaxf(m, lg[h][j]);
      m = warp_max(m);
      float l = 0.f;
      for (int j = lane; j < nk; j += 32) {
        const float e = expf(lg[h][j] - m);
        lg[h][j] = e;
        l += e;
      }
      l = warp_sum(l);
      if (lane == 0) {
        sa[h] = sel ? s_sel[((long long)b * s.Hq + g * G + h) * s.K + u] - logf(l) : m;
        sz[h] = l;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < OUTS; ++r) {
      const int o = tid + r * kThreads;
      if (o >= G * D) continue;
      const int h = o / D, e = o % D;
      float acc = 0.f;
      for (int j = 0; j < nk; ++j) acc = fmaf(lg[h][j], t[j][e], acc);
      float Mh = -INFINITY;
#pragma unroll
      for (int x = 0; x < G; ++x) Mh = x == h ? M[x] : Mh;
      const float Mn = fmaxf(Mh, sa[h]);
      num[r] = num[r] * rel_weight(Mh, Mn) + rel_weight(sa[h], Mn) * (acc * vs);
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float Mn = fmaxf(M[h], sa[h]);
      den[h] = den[h] * rel_weight(M[h], Mn) + rel_weight(sa[h], Mn) * sz[h];
      M[h] = Mn;
    }
  }
#pragma unroll
  for (int r = 0; r < OUTS; ++r) {
    const int o = tid + r * kThreads;
    if (o >= G * D) continue;
    float dh = 1.f;
#pragma unroll
    for (int x = 0; x < G; ++x) dh = x == o / D ? den[x] : dh;
    out[((long long)b * s.Hq + g * G + o / D) * D + o % D] = from_f32<T>(num[r] / dh);
  }
}

template <typename T, typename C, int D, int S, int G>
cudaError_t go_summ(const Shape& s, const CacheView& cv, const DecView& dv, const void* q_lmk, const LmkStrides& ls,
                    const int* from, void* k_sum, float* b_sum, cudaStream_t st, const DevCtx& ctx) {
  if (s.C == 0) return cudaSuccess;
  const size_t smem = sizeof(float) * S * (D + 1);
  auto kern = cache_summaries_kernel<T, C, D, S, G>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, (int)smem);
  if (e != cudaSuccess) return e;
  const int want = (device_sm_count() * 8 + s.B * s.Hkv - 1) / (s.B * s.Hkv);
  kern<<<dim3(want < s.C ? want : s.C, s.Hkv, s.B), kThreads, smem, st>>>(s, cv, dv, (const T*)q_lmk, ls, from,
                                                                          (T*)k_sum, b_sum, ctx);
  return cudaGetLastError();
}

template <typename T, typename C, int D, int S, int G>
cudaError_t go_attn(const Shape& s, const void* q, const CacheView& cv, const DecView& dv, const int32_t* idx,
                    const float* s_sel, void* out, cudaStream_t st, const DevCtx& ctx) {
  const size_t smem = sizeof(float) * S * (D + 1);
  auto kern = attn_codes_kernel<T, C, D, S, G>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(s.Hkv, s.B), kThreads, smem, st>>>(s, (const T*)q, cv, dv, idx, s_sel, (T*)out, ctx);
  return cudaGetLastError();
}

}  // namespace

// F(T, C, d, S, G) for the shape's d, S and G
#define HILS_G(F, T, C, DD, SS, ...)                 \
  if (s.d == DD && s.S == SS) {                      \
    if (s.G == 1) return F<T, C, DD, SS, 1>(__VA_ARGS__); \
    if (s.G == 2) return F<T, C, DD, SS, 2>(__VA_ARGS__); \
    if (s.G == 4) return F<T, C, DD, SS, 4>(__VA_ARGS__); \
    if (s.G == 8) return F<T, C, DD, SS, 8>(__VA_ARGS__); \
  }
// the 8-bit formats' shapes
#define HILS_CODES(F, C, ...)                                                                   \
  if (s.dtype == 0) {                                                                           \
    HILS_G(F, float, C, 64, 32, __VA_ARGS__) HILS_G(F, float, C, 64, 64, __VA_ARGS__)           \
    HILS_G(F, float, C, 128, 32, __VA_ARGS__) HILS_G(F, float, C, 128, 64, __VA_ARGS__)         \
  } else {                                                                                      \
    HILS_G(F, __nv_bfloat16, C, 128, 64, __VA_ARGS__)                                           \
  }

cudaError_t launch_summaries_cache(const Shape& s, const CacheView& cv, const DecView& dv, const void* q_lmk,
                                   const LmkStrides& ls, const int* from, void* k_sum, float* b_sum, cudaStream_t st,
                                   const DevCtx& ctx) {
  if (cv.format == kI8) {
    HILS_CODES(go_summ, int8_t, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
  } else if (cv.format == kE4M3) {
    HILS_CODES(go_summ, __nv_fp8_e4m3, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
  } else if (s.dtype == 0) {
#define HILS_CASE(DD, SS) HILS_G(go_summ, float, float, DD, SS, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
    HILS_CASE(32, 16) HILS_CASE(32, 32) HILS_CASE(64, 16) HILS_CASE(64, 32) HILS_CASE(64, 64)
    HILS_CASE(128, 16) HILS_CASE(128, 32) HILS_CASE(128, 64)
#undef HILS_CASE
  } else {
    HILS_G(go_summ, __nv_bfloat16, __nv_bfloat16, 128, 64, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
  }
  return cudaErrorNotSupported;
}

cudaError_t launch_attn_codes(const Shape& s, const void* q, const CacheView& cv, const DecView& dv,
                              const int32_t* idx, const float* s_sel, void* out, cudaStream_t st, const DevCtx& ctx) {
  if (cv.format == kI8) {
    HILS_CODES(go_attn, int8_t, s, q, cv, dv, idx, s_sel, out, st, ctx)
  } else if (cv.format == kE4M3) {
    HILS_CODES(go_attn, __nv_fp8_e4m3, s, q, cv, dv, idx, s_sel, out, st, ctx)
  }
  return cudaErrorNotSupported;
}

}  // namespace hils
