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
#include "code_mma.cuh"
#include "launch.h"

namespace hils {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Native caches: the summaries on CUDA cores, one CTA for a chunk at a time.
template <typename T, int D, int S, int G>
__global__ void __launch_bounds__(kThreads) native_summaries_kernel(Shape s, CacheView cv, DecView dv,
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
    for (int e = tid; e < S * D; e += kThreads) ks[e / D][e % D] = to_f32(((const T*)cv.k_pool)[off + e]);
    for (int e = tid; e < G * D; e += kThreads) qs[e / D][e % D] = to_f32(q_lmk[ls.of(b, g * G + e / D, c) + e % D]);
    __syncthreads();
    for (int p = tid; p < G * S; p += kThreads) {
      float acc = 0.f;
#pragma unroll 8
      for (int e = 0; e < D; ++e) acc = fmaf(qs[p / S][e], ks[p % S][e], acc);
      lg[p / S][p % S] = acc * s.scale;
    }
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
      k_sum[(((long long)b * s.Hq + g * G + h) * s.C + c) * D + e] = from_f32<T>(acc);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// 8-bit caches: warps work on their own, each on one tile of codes at a time
// (code_mma.cuh), which lane 0 fetches by TMA into the warp's two buffers.
constexpr int kWarps = 4;
constexpr int kCtasPerSm = 3;  // 16 KB of buffers a warp at d = 128, S = 64

template <int D, int S>
struct alignas(1024) WarpBuffers {
  uint8_t a[S * D], b[S * D];
};
// the buffers' start: a multiple of 1024 bytes, as the swizzle counts lines
HILS_DI unsigned char* align_1k(unsigned char* p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }
template <int D, int S>
constexpr size_t buffer_bytes() { return sizeof(WarpBuffers<D, S>) * kWarps + 1024; }
template <int D, int S>
HILS_DI void fetch_tile(void* dst, const CUtensorMap* map, int tile, uint64_t* bar, const DevCtx& ctx) {
  if (ctx.inject == 1) return;  // test hook: no copy, the wait must run out
  mbar_arrive_expect_tx(bar, S * D);
  tma_load_2d(dst, map, 0, tile * (S * D / 128), bar);
}
// pool tile (page Hkv + g) of chunk c of sequence b, or -1: outside the pool (reported)
HILS_DI int dv_tile(const DecView& dv, const Shape& s, int b, int g, int c, const DevCtx& ctx, bool report) {
  const int p = c < dv.max_pages ? __ldg(dv.pages + (long long)b * dv.max_pages + c) : -1;
  if (p >= 0 && p < dv.num_pages) return p * s.Hkv + g;
  if (report) raise_status(ctx, kStatusBadIndex);
  return -1;
}

template <typename T, typename C, int D, int S, int G>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) code_summaries_kernel(
    const __grid_constant__ CUtensorMap kmap, Shape s, CacheView cv, DecView dv, const T* __restrict__ q_lmk,
    LmkStrides ls, const int* __restrict__ from, T* __restrict__ k_sum, float* __restrict__ b_sum, DevCtx ctx) {
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align_1k(smem_raw);
  __shared__ uint64_t bars[kWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c4 = lane & 3;
  const int g = blockIdx.y, b = blockIdx.z;
  WarpBuffers<D, S>& buf = reinterpret_cast<WarpBuffers<D, S>*>(smem)[warp];
  const int L = dv_len(dv, s, b), F = from ? __ldg(from + b) : 0;
  if (L < 1 || L > s.N || F < 0) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && g == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  const int step = gridDim.x * kWarps, end = L / S;
  const int c_first = F / S + blockIdx.x * kWarps + warp;
  if (c_first >= end) return;
  uint64_t* bar = bars[warp];
  if (lane == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  __syncwarp();
  // lane l: tile and scale of the warp's unit l of the next 32
  int my_tile = -1;
  float my_scale = 0.f;
  auto look_up = [&](int c0) {
    const int c = c0 + lane * step;
    my_tile = c < end ? dv_tile(dv, s, b, g, c, ctx, true) : -1;
    my_scale = my_tile >= 0 ? __ldg(cv.k_scale + my_tile) : 0.f;
  };
  look_up(c_first);
  int held = my_tile;  // tiles of units [base, base + 32)
  float held_scale = my_scale;
  int tile = __shfl_sync(0xffffffffu, held, 0);
  if (lane == 0 && tile >= 0) fetch_tile<D, S>(buf.a, &kmap, tile, &bar[0], ctx);
  bool flying[2] = {tile >= 0, false};
  uint32_t phase[2] = {0u, 0u};
  bool alive = true;
  int i = 0;
  for (int c = c_first; c < end; c += step, ++i) {
    const int st = i & 1;
    const float ks = __shfl_sync(0xffffffffu, held_scale, i & 31);
    // the next unit's tile into the other buffer
    int next = -1;
    if (c + step < end) {
      if (((i + 1) & 31) == 0) {
        look_up(c + step);
        held = my_tile;
        held_scale = my_scale;
      }
      next = __shfl_sync(0xffffffffu, held, (i + 1) & 31);
      if (lane == 0 && next >= 0) fetch_tile<D, S>(st ? buf.a : buf.b, &kmap, next, &bar[st ^ 1], ctx);
      flying[st ^ 1] = next >= 0;
    }
    if (tile >= 0) {
      uint32_t qf[PARTS][D / 8];
      const float up = load_qrow<T, C, D, PARTS>(gq < G ? q_lmk + ls.of(b, g * G + gq, c) : nullptr, c4, qf);
      alive = mbar_wait(&bar[st], phase[st], ctx);
      if (!__all_sync(0xffffffffu, alive)) break;
      phase[st] ^= 1u;
      flying[st] = false;
      const uint8_t* t = st ? buf.b : buf.a;
      float sc[S / 16][4], o[D / 16][4];
      tile_scores<C, D, S, PARTS>(t, gq, c4, qf, sc);
      float inv[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int h = 2 * c4 + r;
        const float mul = s.scale * ks * __shfl_sync(0xffffffffu, up, 4 * h);
        float m = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < S / 16; ++mt) {
          sc[mt][r] *= mul;
          sc[mt][2 + r] *= mul;
          m = fmaxf(m, fmaxf(sc[mt][r], sc[mt][2 + r]));
        }
        m = column_max(m);
        if (m == -INFINITY) m = 0.f;
        float z = 0.f, zl = 0.f;
#pragma unroll
        for (int mt = 0; mt < S / 16; ++mt)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            const float l = sc[mt][2 * hi + r] - m, e = weight_of(l);
            sc[mt][2 * hi + r] = e;
            z += e;
            zl += e * l;
          }
        z = column_sum(z);
        zl = column_sum(zl);
        inv[r] = ks / z;
        if (h < G && gq == 0) b_sum[((long long)b * s.Hq + g * G + h) * s.C + c] = logf(z * (1.f / kWeight1)) - zl / z;
      }
      // weights e in half precision (2^-11 of each; float32: two parts), their sum in float32
      tile_values<C, D, S, PARTS>(t, gq, c4, sc, o);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int h = 2 * c4 + r;
        if (h >= G) continue;
        T* dst = k_sum + (((long long)b * s.Hq + g * G + h) * s.C + c) * D + gq * (D / 8);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int v = 0; v < D / 64; ++v)
            *reinterpret_cast<uint4*>(dst + 8 * v) =
                make_uint4(pack_bf16x2(o[4 * v][r] * inv[r], o[4 * v][2 + r] * inv[r]),
                           pack_bf16x2(o[4 * v + 1][r] * inv[r], o[4 * v + 1][2 + r] * inv[r]),
                           pack_bf16x2(o[4 * v + 2][r] * inv[r], o[4 * v + 2][2 + r] * inv[r]),
                           pack_bf16x2(o[4 * v + 3][r] * inv[r], o[4 * v + 3][2 + r] * inv[r]));
        } else {
#pragma unroll
          for (int v = 0; v < D / 32; ++v)
            *reinterpret_cast<float4*>(dst + 4 * v) = make_float4(o[2 * v][r] * inv[r], o[2 * v][2 + r] * inv[r],
                                                                  o[2 * v + 1][r] * inv[r], o[2 * v + 1][2 + r] * inv[r]);
        }
      }
    }
    __syncwarp();  // every lane has read the buffer that the next round refills
    tile = next;
  }
  if (!__all_sync(0xffffffffu, alive) && lane == 0)  // let the copies in flight land before the buffers go
    for (int st = 0; st < 2; ++st)
      if (flying[st] && ctx.inject != 1) mbar_wait(&bar[st], phase[st], ctx);
}

// ------------------------------------------------------------ cluster access ---
HILS_DI void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
HILS_DI float peer_f32(const float* p, int rank) {
  uint32_t a;
  float x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
  return x;
}
// e^{a - M} for a <= M; 0 for a = -inf, also against M = -inf; NaN for a NaN
HILS_DI float rel_weight(float a, float M) { return a == -INFINITY ? 0.f : exp_neg(a - M); }

// eight elements as float32
HILS_DI void row8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
HILS_DI void row8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f32x2(r[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

constexpr int kMaxUnits = 64 + 32;  // K list entries, W / S window chunks

// A cluster of CTAs serves one (sequence, KV head).  Units, dealt to the
// cluster's warps in turn: 16-key slices of the incomplete chunk (in float32 on
// CUDA cores, from the tail), then the window's complete chunks and the chosen
// chunks (tiles of codes).  Each warp folds its units with a running maximum per
// head, the CTA its warps, and the cluster its CTAs through distributed shared
// memory: one launch, no workspace, a fixed order of adding.
template <typename T, typename C, int D, int S, int G>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) attn_codes_kernel(
    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, Shape s,
    const T* __restrict__ q, CacheView cv, DecView dv, const int32_t* __restrict__ idx,
    const float* __restrict__ s_sel, T* __restrict__ out, int ncta, DevCtx ctx) {
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, MT = S / 16, OT = D / 16, N8 = D / 8;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = align_1k(smem_raw);
  __shared__ uint64_t bars[kWarps][2];
  __shared__ int u_tile[kMaxUnits], u_slot[kMaxUnits], n_units;
  __shared__ float u_ks[kMaxUnits], u_vs[kMaxUnits];
  __shared__ float red_m[kWarps][G], red_d[kWarps][G], cta_m[G], cta_d[G];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c4 = lane & 3;
  const int rank = blockIdx.x % ncta, g = (int)(blockIdx.x / ncta) % s.Hkv, b = (int)(blockIdx.x / ncta) / s.Hkv;
  const int L = dv_len(dv, s, b);
  if (L < 1 || L > s.N) {  // the whole cluster: reported, nothing written
    if (rank == 0 && threadIdx.x == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  const int cur = (L - 1) / S, wc0 = max(0, cur - s.nw + 1);
  const int n_full = L / S - wc0, part = L % S, n_tail = (part + 15) / 16;
  uint64_t* bar = bars[warp];
  if (lane == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  const T* q0 = q + ((long long)b * s.Hq + g * G) * D;
  uint32_t qf[PARTS][D / 8];
  float qmul[2];
  if (warp == 0) {
    // the live units: window chunks, then accepted list entries (the list form, common.cuh)
    const int32_t* ir = idx + ((long long)b * s.Hkv + g) * s.K;
    int e0 = lane < s.K ? __ldg(ir + lane) : -1, e1 = lane + 32 < s.K ? __ldg(ir + lane + 32) : -1;
    bool bad;
    accept_list_warp(e0, e1, s.K, wc0, bad);
    if (bad && lane == 0 && rank == 0) raise_status(ctx, kStatusBadIndex);
    const int c[3] = {lane < n_full ? wc0 + lane : -1, e0, e1};
    int n = 0;
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const int tile = c[x] >= 0 ? dv_tile(dv, s, b, g, c[x], ctx, rank == 0) : -1;
      const unsigned live = __ballot_sync(0xffffffffu, tile >= 0);
      if (tile >= 0) {
        const int at = n + __popc(live & ((1u << lane) - 1u));
        u_tile[at] = tile;
        u_slot[at] = x == 0 ? -1 : lane + 32 * (x - 1);
        u_ks[at] = __ldg(cv.k_scale + tile);
        u_vs[at] = __ldg(cv.v_scale + tile);
      }
      n += __popc(live);
    }
    if (lane == 0) n_units = n;
  }
  {
    const float up = load_qrow<T, C, D, PARTS>(gq < G ? q0 + gq * D : nullptr, c4, qf);
#pragma unroll
    for (int r = 0; r < 2; ++r) qmul[r] = s.scale * __shfl_sync(0xffffffffu, up, 4 * (2 * c4 + r));
  }
  __syncthreads();

  WarpBuffers<D, S>& buf = reinterpret_cast<WarpBuffers<D, S>*>(smem)[warp];
  const int step = ncta * kWarps, end = n_units + n_tail;
  int i = rank * kWarps + warp;
  int first = i;  // the warp's first unit of codes
  while (first < n_tail) first += step;
  bool flying[2] = {false, false};
  uint32_t phase[2] = {0u, 0u};
  bool alive = true;
  if (first < end) {
    if (lane == 0) {
      fetch_tile<D, S>(buf.a, &kmap, u_tile[first - n_tail], &bar[0], ctx);
      fetch_tile<D, S>(buf.b, &vmap, u_tile[first - n_tail], &bar[1], ctx);
    }
    flying[0] = flying[1] = true;
  }

  float acc[OT][4], M[2] = {-INFINITY, -INFINITY}, den[2] = {0.f, 0.f};
#pragma unroll
  for (int mt = 0; mt < OT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
  // weights of a unit against the running maximum: fo for what is there, fu for the unit
  auto fold = [&](int r, float lam, float mass, float& fo, float& fu) {
    const float Mn = fmaxf(M[r], lam);
    fo = rel_weight(M[r], Mn);
    fu = rel_weight(lam, Mn);
    den[r] = den[r] * fo + fu * mass;
    M[r] = Mn;
  };

  for (; i < n_tail; i += step) {
    // keys [16 i, 16 i + 16) of the incomplete chunk, in float32
    const long long off = tail_off(s, b, g, cur) + 16 * i * D;
    const T* kt = (const T*)cv.k_tail + off;
    const T* vt = (const T*)cv.v_tail + off;
    const int nk = min(16, part - 16 * i);
    float sc[4] = {0.f, 0.f, 0.f, 0.f};  // key gq: columns 2 c4, 2 c4 + 1; key gq + 8
#pragma unroll 4
    for (int e = 0; e < D; e += 8) {
      float k0[8], k1[8], qa[8], qb[8];
      row8(kt + min(gq, nk - 1) * D + e, k0);
      row8(kt + min(gq + 8, nk - 1) * D + e, k1);
      row8(q0 + min(2 * c4, G - 1) * D + e, qa);
      row8(q0 + min(2 * c4 + 1, G - 1) * D + e, qb);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        sc[0] = fmaf(k0[x], qa[x], sc[0]);
        sc[1] = fmaf(k0[x], qb[x], sc[1]);
        sc[2] = fmaf(k1[x], qa[x], sc[2]);
        sc[3] = fmaf(k1[x], qb[x], sc[3]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sc[r] = gq < nk ? sc[r] * s.scale : -INFINITY;
      sc[2 + r] = gq + 8 < nk ? sc[2 + r] * s.scale : -INFINITY;
      const float top = column_max(fmaxf(sc[r], sc[2 + r])), m = top == -INFINITY ? 0.f : top;
      sc[r] = exp_neg(sc[r] - m);
      sc[2 + r] = exp_neg(sc[2 + r] - m);
      float fo, fu;
      fold(r, top, column_sum(sc[r] + sc[2 + r]), fo, fu);
      sc[r] *= fu;
      sc[2 + r] *= fu;
#pragma unroll
      for (int mt = 0; mt < OT; ++mt) acc[mt][r] *= fo, acc[mt][2 + r] *= fo;
    }
#pragma unroll 4
    for (int k = 0; k < nk; ++k) {
      const float p0 = __shfl_sync(0xffffffffu, k < 8 ? sc[0] : sc[2], 4 * (k & 7) + c4);
      const float p1 = __shfl_sync(0xffffffffu, k < 8 ? sc[1] : sc[3], 4 * (k & 7) + c4);
#pragma unroll
      for (int e = 0; e < N8; e += 8) {
        float v[8];
        row8(vt + k * D + gq * N8 + e, v);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int mt = (e + x) / 2, hi = 2 * (x & 1);
          acc[mt][hi] = fmaf(p0, v[x], acc[mt][hi]);
          acc[mt][hi + 1] = fmaf(p1, v[x], acc[mt][hi + 1]);
        }
      }
    }
  }

  for (i = first; i < end; i += step) {
    const int u = i - n_tail, next = i + step < end ? u_tile[u + step] : -1, slot = u_slot[u];
    const float ks = u_ks[u], vs = u_vs[u];
    float shat[2] = {0.f, 0.f};
    if (slot >= 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (2 * c4 + r < G) shat[r] = __ldg(s_sel + ((long long)b * s.Hq + g * G + 2 * c4 + r) * s.K + slot);
    }
    float sc[MT][4], o[OT][4];
    alive = mbar_wait(&bar[0], phase[0], ctx);
    if (!__all_sync(0xffffffffu, alive)) break;
    flying[0] = false;
    phase[0] ^= 1u;
    tile_scores<C, D, S, PARTS>(buf.a, gq, c4, qf, sc);
    __syncwarp();  // every lane has read the keys: their buffer takes the next unit's
    if (next >= 0) {
      if (lane == 0) fetch_tile<D, S>(buf.a, &kmap, next, &bar[0], ctx);
      flying[0] = true;
    }
    float fo[2], fu[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float mul = qmul[r] * ks;
      float top = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        sc[mt][r] *= mul;
        sc[mt][2 + r] *= mul;
        top = fmaxf(top, fmaxf(sc[mt][r], sc[mt][2 + r]));
      }
      top = column_max(top);
      const float m = top == -INFINITY ? 0.f : top;
      float l = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        sc[mt][r] = weight_of(sc[mt][r] - m);
        sc[mt][2 + r] = weight_of(sc[mt][2 + r] - m);
        l += sc[mt][r] + sc[mt][2 + r];
      }
      l = column_sum(l);  // of weights times 2^15
      // a chosen chunk weighs e^{s^} whatever its l; a window chunk e^{top} l
      fold(r, slot >= 0 ? shat[r] : top, slot >= 0 ? 1.f : l * (1.f / kWeight1), fo[r], fu[r]);
      fu[r] *= slot >= 0 ? vs / l : vs * (1.f / kWeight1);
    }
    alive = mbar_wait(&bar[1], phase[1], ctx);
    if (!__all_sync(0xffffffffu, alive)) break;
    flying[1] = false;
    phase[1] ^= 1u;
    tile_values<C, D, S, PARTS>(buf.b, gq, c4, sc, o);
    __syncwarp();
    if (next >= 0) {
      if (lane == 0) fetch_tile<D, S>(buf.b, &vmap, next, &bar[1], ctx);
      flying[1] = true;
    }
#pragma unroll
    for (int mt = 0; mt < OT; ++mt)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[mt][x] = acc[mt][x] * fo[x & 1] + o[mt][x] * fu[x & 1];
  }
  if (!__all_sync(0xffffffffu, alive) && lane == 0 && ctx.inject != 1) {
    // a wait ran out: let the copies in flight land before the buffers change hands
    if (flying[0]) mbar_wait(&bar[0], phase[0], ctx);
    if (flying[1]) mbar_wait(&bar[1], phase[1], ctx);
  }
  __syncthreads();  // every warp's copies have landed and been read: the buffers now hold the records

  float* rec = reinterpret_cast<float*>(smem);
  float* cta = rec + kWarps * G * D;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int h = 2 * c4 + r;
    if (h >= G) continue;
#pragma unroll
    for (int mt = 0; mt < OT; ++mt)
      *reinterpret_cast<float2*>(rec + (warp * G + h) * D + gq * N8 + 2 * mt) = make_float2(acc[mt][r], acc[mt][2 + r]);
    if (gq == 0) {
      red_m[warp][h] = M[r];
      red_d[warp][h] = den[r];
    }
  }
  __syncthreads();
  T* o0 = out + ((long long)b * s.Hq + g * G) * D;
  for (int x = threadIdx.x; x < G * D; x += kWarps * 32) {
    const int h = x / D;
    float Mx = red_m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) Mx = fmaxf(Mx, red_m[w][h]);
    float num = 0.f, dd = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = rel_weight(red_m[w][h], Mx);
      num += f * rec[w * G * D + x];
      dd += f * red_d[w][h];
    }
    if (ncta == 1) {
      o0[x] = from_f32<T>(num / dd);
    } else {
      cta[x] = num;
      if (x % D == 0) {
        cta_m[h] = Mx;
        cta_d[h] = dd;
      }
    }
  }
  if (ncta == 1) return;
  cluster_sync();
  for (int x = rank * kWarps * 32 + threadIdx.x; x < G * D; x += ncta * kWarps * 32) {
    const int h = x / D;
    float Mx = -INFINITY;
    for (int w = 0; w < ncta; ++w) Mx = fmaxf(Mx, peer_f32(&cta_m[h], w));
    float num = 0.f, dd = 0.f;
    for (int w = 0; w < ncta; ++w) {
      const float f = rel_weight(peer_f32(&cta_m[h], w), Mx);
      num += f * peer_f32(cta + x, w);
      dd += f * peer_f32(&cta_d[h], w);
    }
    o0[x] = from_f32<T>(num / dd);
  }
  cluster_sync();  // no CTA leaves while its records are read
}

template <typename T, typename C, int D, int S, int G>
cudaError_t go_summ(const Shape& s, const CacheView& cv, const DecView& dv, const void* q_lmk, const LmkStrides& ls,
                    const int* from, void* k_sum, float* b_sum, cudaStream_t st, const DevCtx& ctx) {
  if (s.C == 0) return cudaSuccess;
  const size_t smem = buffer_bytes<D, S>();
  auto kern = code_summaries_kernel<T, C, D, S, G>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, (int)smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km;
  e = make_tmap_rows128(&km, cv.k_pool, (uint64_t)dv.num_pages * s.Hkv * (S * D / 128), S * D / 128);
  if (e != cudaSuccess) return e;
  const int most = (s.C + kWarps - 1) / kWarps;
  const int want = (device_sm_count() * kCtasPerSm * 2 + s.B * s.Hkv - 1) / (s.B * s.Hkv);
  kern<<<dim3(want < most ? want : most, s.Hkv, s.B), kWarps * 32, smem, st>>>(km, s, cv, dv, (const T*)q_lmk, ls, from,
                                                                                (T*)k_sum, b_sum, ctx);
  return cudaGetLastError();
}

template <typename T, int D, int S, int G>
cudaError_t go_native(const Shape& s, const CacheView& cv, const DecView& dv, const void* q_lmk, const LmkStrides& ls,
                      const int* from, void* k_sum, float* b_sum, cudaStream_t st, const DevCtx& ctx) {
  if (s.C == 0) return cudaSuccess;
  const size_t smem = sizeof(float) * S * (D + 1);
  auto kern = native_summaries_kernel<T, D, S, G>;
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
  const size_t smem = buffer_bytes<D, S>();
  static_assert(sizeof(float) * (kWarps + 1) * G * D <= sizeof(WarpBuffers<D, S>) * kWarps, "records fit the buffers");
  auto kern = attn_codes_kernel<T, C, D, S, G>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, (int)smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)dv.num_pages * s.Hkv * (S * D / 128);
  e = make_tmap_rows128(&km, cv.k_pool, rows, S * D / 128);
  if (e == cudaSuccess) e = make_tmap_rows128(&vm, cv.v_pool, rows, S * D / 128);
  if (e != cudaSuccess) return e;
  // CTAs of a cluster: as many as fit the device at once, and no more than there are units for
  const int groups = s.B * s.Hkv, units = s.K + s.nw + 3;
  int ncta = device_sm_count() * kCtasPerSm / groups;
  ncta = ncta > 8 ? 8 : ncta;
  ncta = ncta > (units + kWarps - 1) / kWarps ? (units + kWarps - 1) / kWarps : ncta;
  ncta = ncta < 1 ? 1 : ncta;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)groups * ncta);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ncta;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, km, vm, s, (const T*)q, cv, dv, idx, s_sel, (T*)out, ncta, ctx);
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
#define HILS_N(T, DD, SS, ...)                       \
  if (s.d == DD && s.S == SS) {                      \
    if (s.G == 1) return go_native<T, DD, SS, 1>(__VA_ARGS__); \
    if (s.G == 2) return go_native<T, DD, SS, 2>(__VA_ARGS__); \
    if (s.G == 4) return go_native<T, DD, SS, 4>(__VA_ARGS__); \
    if (s.G == 8) return go_native<T, DD, SS, 8>(__VA_ARGS__); \
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
    HILS_CODES(go_summ, CodeI8, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
  } else if (cv.format == kE4M3) {
    HILS_CODES(go_summ, CodeE4M3, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
  } else {
#define HILS_CASE(T, DD, SS) HILS_N(T, DD, SS, s, cv, dv, q_lmk, ls, from, k_sum, b_sum, st, ctx)
    if (s.dtype == 0) {
      HILS_CASE(float, 32, 16) HILS_CASE(float, 32, 32) HILS_CASE(float, 64, 16) HILS_CASE(float, 64, 32)
      HILS_CASE(float, 64, 64) HILS_CASE(float, 128, 16) HILS_CASE(float, 128, 32) HILS_CASE(float, 128, 64)
    } else {
      HILS_CASE(__nv_bfloat16, 128, 64)
    }
#undef HILS_CASE
  }
  return cudaErrorNotSupported;
}

cudaError_t launch_attn_codes(const Shape& s, const void* q, const CacheView& cv, const DecView& dv,
                              const int32_t* idx, const float* s_sel, void* out, cudaStream_t st, const DevCtx& ctx) {
  if (cv.format == kI8) {
    HILS_CODES(go_attn, CodeI8, s, q, cv, dv, idx, s_sel, out, st, ctx)
  } else if (cv.format == kE4M3) {
    HILS_CODES(go_attn, CodeE4M3, s, q, cv, dv, idx, s_sel, out, st, ctx)
  }
  return cudaErrorNotSupported;
}

}  // namespace hils
