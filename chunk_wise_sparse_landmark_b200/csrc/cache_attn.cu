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
#include <cfloat>

#include "code_mma.cuh"
#include "launch.h"

namespace hils {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Native caches: the summaries on CUDA cores, one CTA for a chunk at a time: 131072
// tokens, 32 heads over 8, bf16: 300 us for a floor of 46; 32768 in float32, d = 64,
// 16 heads over 4: 23 us for 6.4 (hils_build_summaries_paged: 299, 25).  Far from
// the memory's rate: scalar products out of shared memory, two-byte loads.
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
// (code_mma.cuh), which lane 0 fetches by TMA into the warp's buffers.
constexpr int kWarps = 4;  // of a CTA that builds summaries

template <int D, int S>
struct alignas(1024) WarpBuffers {
  uint8_t a[S * D], b[S * D];
};
// the buffers' start: a multiple of 1024 bytes, as the swizzle counts lines
HILS_DI unsigned char* align_1k(unsigned char* p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }
template <int D, int S>
HILS_DI Tile<D, S> tile_of(const uint8_t* p) { return Tile<D, S>{{p, p + S * D / 2}}; }
template <int D, int S>
HILS_DI void fetch_tile(void* dst, const CUtensorMap* map, int tile, uint64_t* bar, const DevCtx& ctx) {
  if (ctx.inject == 1) return;  // test hook: no copy, the wait must run out
  mbar_arrive_expect_tx(bar, S * D);
  tma_load_2d(dst, map, 0, tile * (S * D / 128), bar);
}
HILS_DI void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
// pool tile (page Hkv + g) of chunk c of sequence b, or -1: outside the pool (reported)
HILS_DI int dv_tile(const DecView& dv, const Shape& s, int b, int g, int c, const DevCtx& ctx, bool report) {
  const int p = c < dv.max_pages ? __ldg(dv.pages + (long long)b * dv.max_pages + c) : -1;
  if (p >= 0 && p < dv.num_pages) return p * s.Hkv + g;
  if (report) raise_status(ctx, kStatusBadIndex);
  return -1;
}

// which of code_mma.cuh's functions (measured there)
template <typename T, typename C, int D, int S, int G>
struct OpsOf {
  using type = HalfOps<C, D, S, G, sizeof(T) == 4 ? 2 : 1>;
};
template <int D, int S>
struct OpsOf<__nv_bfloat16, CodeI8, D, S, 1> {
  using type = DigitOps<D, S, 1>;
};
template <int D, int S>
struct OpsOf<__nv_bfloat16, CodeI8, D, S, 2> {
  using type = DigitOps<D, S, 2>;
};
template <int D, int S>
struct OpsOf<__nv_bfloat16, CodeI8, D, S, 4> {
  using type = DigitOps<D, S, 4>;
};

// sc (scores) -> weights kOne e^{x - top} of the logits x = sc mul: `top` the
// column's largest logit, `l` the weights' sum (float32); zl, if wanted, the sum of
// weight * (x - top).  The largest score is taken off before the scaling: its own
// exponent is 0 whatever the logits' size, so that no weight is above kOne, which
// the digits and halves of the products (code_mma.cuh) have little room beyond.  (One
// instruction a weight: 131072 tokens' summaries 35.2 us for 35.0, attention 81.2 for 80.9.)
template <typename Ops, int N>
HILS_DI void weigh(float (&sc)[N], float mul, float& top, float& l, float* zl = nullptr) {
  if (mul < 0.f) {  // (a scale of a pool that was filled elsewhere)
    mul = -mul;
#pragma unroll
    for (int i = 0; i < N; ++i) sc[i] = -sc[i];
  }
  float m = sc[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, sc[i]);
  m = column_max(m);
  top = m * mul;
  const float f = mul * kLog2e, c = m == -INFINITY ? 0.f : m;
  l = 0.f;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (zl) {
      const float x = (sc[i] - c) * f;
      sc[i] = exp2_fast(x + Ops::kLog2One);
      z = fmaf(sc[i], x, z);
    } else {
      sc[i] = exp2_fast(fmaf(sc[i] - c, f, Ops::kLog2One));
    }
    l += sc[i];
  }
  l = column_sum(l);
  if (zl) *zl = column_sum(z) * kLn2;
}

// A block's scale over a sum of weights (up to 2^21) may fall below the normal
// range where the block's values do not: such a scale is multiplied by 2^40 and the
// block's sums by 2^-40.
template <int R, int N>
HILS_DI float lift(float scale, float (&o)[R][N]) {
  if (fabsf(scale) >= 0x1p-90f || scale != scale) return scale;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int x = 0; x < N; ++x) o[r][x] *= 0x1p-40f;
  return scale * 0x1p40f;
}

// Warps take the chunks of all sequences in turn, so that short and long
// sequences share the work evenly.  A CTA serves sequences [kSeqs blockIdx.y, +
// kSeqs): their numbers of chunks are summed up in shared memory, and unit u is
// KV head u % Hkv of chunk u / Hkv of that order.  The latency of a warp's own chain
// bounds it, about 1100 instructions for a tile of 8 KB, most of them waiting for one
// just before (issue slots 53% used, ALU pipe 50%, tensor pipe 24%; without its tile copies it
// takes as long), so that many warps matter: a warp has three half tiles of buffer,
// 12 KB, and sixteen warps share a multiprocessor (two whole tiles and twelve warps:
// 39.6 us instead of 35.2).  It holds a tile and the first half of the next one, whose
// second half takes the place of this one's first half once that has been read.
// The landmark rows of the next unit are asked for before this one is computed.
// 131072 tokens, 32 heads over 8, e4m3: 34.8 us, 4.8 TB/s of the 168 MB it must move;
// 55K tokens in 13 sequences, 16 heads over 8, int8: 17.7 us, 3.6 TB/s.
constexpr int kSeqs = 512;
template <typename T>
constexpr int summary_ctas() { return sizeof(T) == 2 ? 4 : 3; }  // of a multiprocessor
template <int D, int S>
struct alignas(1024) HalfTiles {
  uint8_t h[3][S * D / 2];
};

template <typename T, typename C, int D, int S, int G>
__global__ void __launch_bounds__(kWarps * 32, summary_ctas<T>()) code_summaries_kernel(
    const __grid_constant__ CUtensorMap kmap, Shape s, CacheView cv, DecView dv, const T* q_lmk,
    LmkStrides ls, const int* from, T* k_sum, float* b_sum, DevCtx ctx) {
  using Ops = typename OpsOf<T, C, D, S, G>::type;
  constexpr int R = Ops::R, N8 = D / 8;
  constexpr int PER = kSeqs / (kWarps * 32);  // sequences of a thread
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[kWarps][3];
  __shared__ int ends[kSeqs], firsts[kSeqs], sums[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, c4 = lane & 3;
  const int b0 = blockIdx.y * kSeqs, nb = min(kSeqs, s.B - b0);
  HalfTiles<D, S>& buf = reinterpret_cast<HalfTiles<D, S>*>(align_1k(smem_raw))[warp];
  uint64_t* bar = bars[warp];
  if (lane == 0) {
    prefetch_tmap(&kmap);
#pragma unroll
    for (int x = 0; x < 3; ++x) mbar_init(&bar[x], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  const unsigned long long zero = grid_begin();
  behind(zero, cv), behind(zero, dv), behind(zero, q_lmk), behind(zero, from);
  if (lane == 0) fence_proxy_async_all();  // what earlier kernels stored is read by tile copies
  // chunks up to and with each sequence
  int n[PER], own = 0;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int b = tid * PER + x;
    n[x] = 0;
    if (b < nb) {
      const int L = dv_len(dv, s, b0 + b), F = from ? __ldg(from + b0 + b) : 0;
      const bool ok = L >= 1 && L <= s.N && F >= 0;
      if (!ok && blockIdx.x == 0) raise_status(ctx, kStatusBadIndex);
      firsts[b] = F / S;
      n[x] = ok ? max(0, L / S - F / S) : 0;
    }
    own += n[x];
  }
  int upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += sums[w];
    total += sums[w];
  }
  upto -= own;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    upto += n[x];
    if (tid * PER + x < nb) ends[tid * PER + x] = upto;
  }
  __syncthreads();
  const long long units = (long long)total * s.Hkv, step = (long long)gridDim.x * kWarps;
  long long u = (long long)blockIdx.x * kWarps + warp;
  if (u >= units) return;
  const TileOffsets<D> at(gq, c4);

  // lane l: sequence, chunk, tile and scale of the warp's unit l of the next 32
  int my_b = 0, my_c = 0, my_g = 0, my_tile = -1;
  float my_scale = 0.f;
  auto look_up = [&](long long u0) {
    const long long v = u0 + lane * step;
    my_tile = -1;
    if (v < units) {
      const int t = (int)(v / s.Hkv);
      my_g = (int)(v - (long long)t * s.Hkv);
      int lo = 0, hi = nb - 1;  // the first sequence that ends behind t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
      }
      my_b = b0 + lo;
      my_c = firsts[lo] + t - (lo ? ends[lo - 1] : 0);
      my_tile = dv_tile(dv, s, my_b, my_g, my_c, ctx, true);
    }
    my_scale = my_tile >= 0 ? __ldg(cv.k_scale + my_tile) : 0.f;
  };
  struct Unit {
    int b, g, c, tile;
    float ks;  // filled in by scale_of, behind the tile's fetch
  };
  auto unit_of = [&](int i) {
    Unit x;
    x.b = __shfl_sync(0xffffffffu, my_b, i & 31);
    x.g = __shfl_sync(0xffffffffu, my_g, i & 31);
    x.c = __shfl_sync(0xffffffffu, my_c, i & 31);
    x.tile = __shfl_sync(0xffffffffu, my_tile, i & 31);
    return x;
  };
  auto scale_of = [&](int i) { return __shfl_sync(0xffffffffu, my_scale, i & 31); };
  const int row = Ops::row_head(gq);
  auto ask_query = [&](const Unit& x, RawRow<T, D>& raw) {
    raw.load(row < G ? q_lmk + ls.of(x.b, x.g * G + row, x.c) : (const T*)nullptr, c4);
  };
  // Half tiles n = 0, 1, 2 .. (two to a unit) go to buffers n % 3.  A unit whose
  // page is outside the pool is fetched as tile 0 and left out.
  int n_asked = 0;  // half tiles asked for
  auto ask_half = [&](int tile) {
    const int slot = n_asked % 3, half = n_asked & 1;
    if (lane == 0 && ctx.inject != 1) {  // (test hook: no copy, the wait must run out)
      mbar_arrive_expect_tx(&bar[slot], S * D / 2);
      tma_load_2d(buf.h[slot], &kmap, 0, max(tile, 0) * (S * D / 128) + half * (S * D / 256), &bar[slot]);
    }
    ++n_asked;
  };
  look_up(u);
  Unit now = unit_of(0), next;
  ask_half(now.tile);
  ask_half(now.tile);
  RawRow<T, D> raw;
  ask_query(now, raw);
  next.tile = -1;
  if (u + step < units) {
    next = unit_of(1);
    ask_half(next.tile);
    next.ks = scale_of(1);
  }
  now.ks = scale_of(0);
  bool alive = true;
  int i = 0;
  for (; u < units; u += step, ++i) {
    const bool more = u + step < units;
    // behind the next unit: its first half follows this unit's second half
    Unit later;
    later.tile = -1;
    const bool more2 = u + 2 * step < units;
    if (more2) {
      if (((i + 2) & 31) == 0) look_up(u + 2 * step);
      later = unit_of(i + 2);
      later.ks = scale_of(i + 2);
    }
    typename Ops::Query q;
    Ops::template make_query<T>(raw, gq, c4, q);
    if (more) ask_query(next, raw);
    const int n0 = 2 * i, s0 = n0 % 3, s1 = (n0 + 1) % 3;
    alive = mbar_wait(&bar[s0], (n0 / 3) & 1, ctx) && mbar_wait(&bar[s1], ((n0 + 1) / 3) & 1, ctx);
    if (!__all_sync(0xffffffffu, alive)) break;
    {
      const Tile<D, S> t{{buf.h[s0], buf.h[s1]}};
      float sc[R][S / 8], o[R][N8], zs[R], zls[R];
      Ops::scores(t, at, q, sc);
      const long long h0 = (long long)now.b * s.Hq + now.g * G;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float top;
        weigh<Ops>(sc[r], s.scale * now.ks * q.up[r], top, zs[r], &zls[r]);
      }
      // lane gq = r of a column writes the entropy of its head r: log l - (sum of weight x) / l
      if (gq < R) {
        const int h = Ops::head(gq, c4);
        const float z = gq == 0 ? zs[0] : zs[R - 1], zl = gq == 0 ? zls[0] : zls[R - 1];
        if (h < G && now.tile >= 0)
          b_sum[(h0 + h) * s.C + now.c] = kLn2 * __log2f(z * (1.f / Ops::kOne)) - __fdividef(zl, z);
      }
      Ops::values(t, at, gq, sc, o, [&] {
        __syncwarp();  // every lane has read the first half
        if (more) ask_half(next.tile);
      });
      const float ks = lift(now.ks, o);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = Ops::head(r, c4);
        const float inv = __fdividef(ks, zs[r]);
        if (h >= G || now.tile < 0) continue;
        T* dst = k_sum + ((h0 + h) * s.C + now.c) * D + gq * N8;
#pragma unroll
        for (int x = 0; x < N8; ++x) o[r][x] *= inv;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int x = 0; x < N8; x += 8)
            *reinterpret_cast<uint4*>(dst + x) =
                make_uint4(pack_bf16x2(o[r][x], o[r][x + 1]), pack_bf16x2(o[r][x + 2], o[r][x + 3]),
                           pack_bf16x2(o[r][x + 4], o[r][x + 5]), pack_bf16x2(o[r][x + 6], o[r][x + 7]));
        } else {
#pragma unroll
          for (int x = 0; x < N8; x += 4)
            *reinterpret_cast<float4*>(dst + x) = make_float4(o[r][x], o[r][x + 1], o[r][x + 2], o[r][x + 3]);
        }
      }
    }
    __syncwarp();  // every lane has read the second half
    if (more2) ask_half(later.tile);
    now = next;
    next = later;
  }
  if (!__all_sync(0xffffffffu, alive) && lane == 0 && ctx.inject != 1)  // let the copies in flight land first
    for (int n = 2 * i; n < n_asked; ++n) mbar_wait(&bar[n % 3], (n / 3) & 1, ctx);
}

// ------------------------------------------------------------ cluster access ---
HILS_DI void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
HILS_DI void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// into the shared memory of the cluster's first CTA, where `p` is in this one's
HILS_DI void store_first(float* p, float x) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
HILS_DI void store_first(float* p, const float4& x) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
               : "memory");
}
// A running maximum starts at -inf and is compared as no less than kLeast, the
// least finite number, so that e^{a - M} is 0 for a = -inf (and NaN for a NaN)
// without a case of its own.
constexpr float kLeast = -FLT_MAX;
HILS_DI float max_of(float a, float b) { return fmaxf(fmaxf(a, b), kLeast); }

// eight elements as float32
HILS_DI void row8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// KEYS keys of a tail, with the arithmetic of float32: scores sc[r][x] of key
// gq + 8 x and head Ops::head(r, c4), and acc += weights . values (dims gq D / 8 + x).
// float32 configurations: on CUDA cores, eight keys, so that a tail is shared by more
// warps, and a quarter of a key's dims to a thread (24 sequences of 4K, d = 64, S = 32,
// G = 4: 7.5 us; sixteen keys 10.3; eight, a key's dims and two heads to a thread 7.9).
template <typename T, typename Ops, int D>
struct TailSlice {
  static constexpr int R = Ops::R, N8 = D / 8, KEYS = 8;
  HILS_DI static void f4(const float* p, float* y) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w;
  }
  const T *kt, *vt, *q0;
  int nk, heads, gq, c4;
  HILS_DI void load(const T* kt_, const T* vt_, const T* q0_, int nk_, int G, int gq_, int c4_) {
    kt = kt_, vt = vt_, q0 = q0_, nk = nk_, heads = G, gq = gq_, c4 = c4_;
  }
  // key gq, the dims 16 e + 4 c4 .., + 3, all heads; then the quarters are added
  HILS_DI void scores(float (&sc)[R][KEYS / 8]) const {
    const T* kr = kt + min(gq, nk - 1) * D;
    float x[D / 4];
#pragma unroll
    for (int e = 0; e < D / 4; e += 4) f4(kr + 4 * e + 4 * c4, x + e);
    sc[0][0] = sc[R - 1][0] = 0.f;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      if (h >= heads) break;
      const T* qr = q0 + h * D + 4 * c4;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < D / 4; e += 4) {
        float y[4];
        f4(qr + 4 * e, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fmaf(x[e + i], y[i], sum);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
      for (int r = 0; r < R; ++r) sc[r][0] = h == Ops::head(r, c4) ? sum : sc[r][0];
    }
  }
  HILS_DI void add_values(const float (&p)[R][KEYS / 8], float (&acc)[R][N8]) const {
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      float w[R];
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = __shfl_sync(0xffffffffu, p[r][0], 4 * k + c4);
#pragma unroll
      for (int e = 0; e < N8; e += 8) {
        float v[8];
        row8(vt + min(k, nk - 1) * D + gq * N8 + e, v);
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = k < nk ? v[x] : 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[r][e + x] = fmaf(w[r], v[x], acc[r][e + x]);
      }
    }
  }
};
HILS_DI float bf16_part(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
// bf16 configurations: bf16 mma.sync, all of the slice's loads in flight at once.
// Weights are the sum of two bf16 numbers (within 2^-17 of themselves), as two
// products, or where a thread has one head, in the two columns of that head.
template <typename Ops, int D>
struct TailSlice<__nv_bfloat16, Ops, D> {
  using T = __nv_bfloat16;
  static constexpr int R = Ops::R, N8 = D / 8, KEYS = 16, Q4 = D / 32, V4 = N8 / 8;
  uint4 k[2][Q4], q[Q4], v[4][V4];
  HILS_DI static uint32_t word(const uint4* x, int i) {
    const uint4& w = x[i >> 2];
    return (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w;
  }
  HILS_DI void load(const T* kt, const T* vt, const T* q0, int nk, int G, int gq, int c4) {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const int h = Ops::row_head(gq);
#pragma unroll
    for (int x = 0; x < Q4; ++x) {
      k[0][x] = __ldg(reinterpret_cast<const uint4*>(kt + min(gq, nk - 1) * D + c4 * (D / 4)) + x);
      k[1][x] = __ldg(reinterpret_cast<const uint4*>(kt + min(gq + 8, nk - 1) * D + c4 * (D / 4)) + x);
      q[x] = h < G ? __ldg(reinterpret_cast<const uint4*>(q0 + h * D + c4 * (D / 4)) + x) : none;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = 2 * c4 + (e & 1) + 8 * (e >> 1);
#pragma unroll
      for (int x = 0; x < V4; ++x)
        v[e][x] = key < nk ? __ldg(reinterpret_cast<const uint4*>(vt + key * D + gq * N8) + x) : none;
    }
  }
  HILS_DI void scores(float (&sc)[R][2]) const {
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t A[4] = {word(k[0], 2 * ks), word(k[1], 2 * ks), word(k[0], 2 * ks + 1), word(k[1], 2 * ks + 1)};
      mma_bf16_16816(d, A, word(q, 2 * ks), word(q, 2 * ks + 1));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) sc[r][0] = d[r], sc[r][1] = d[2 + r];
  }
  HILS_DI void add_values(const float (&p)[R][2], float (&acc)[R][N8]) const {
    uint32_t b[2][R];
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const float x0 = p[0][hi], x1 = R == 2 ? p[R - 1][hi] : x0 - bf16_part(x0);
      b[hi][0] = movmatrix_trans16(pack_bf16x2(x0, x1));
      if (R == 2) b[hi][R - 1] = movmatrix_trans16(pack_bf16x2(x0 - bf16_part(x0), x1 - bf16_part(x1)));
    }
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const uint32_t w[4] = {word(v[0], mt), word(v[1], mt), word(v[2], mt), word(v[3], mt)};
      const uint32_t A[4] = {__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                             __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632)};
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < R; ++x) mma_bf16_16816(d, A, b[0][x], b[1][x]);
      if (R == 2) {
        acc[0][2 * mt] += d[0], acc[R - 1][2 * mt] += d[1];
        acc[0][2 * mt + 1] += d[2], acc[R - 1][2 * mt + 1] += d[3];
      } else {
        acc[0][2 * mt] += d[0] + d[1];
        acc[0][2 * mt + 1] += d[2] + d[3];
      }
    }
  }
};

constexpr int kMaxUnits = 64 + 32;  // K list entries, W / S window chunks
constexpr int kMaxCtas = 8;         // of a cluster
constexpr int kMaxWarps = 12;       // 16 KB of buffers each at d = 128, S = 64, up to 170 registers a thread
constexpr int kMaxWarpsOfMany = 10;  // beside the records of a cluster's CTAs
// a CTA's record: sums [G][D], then for each head its reference and denominator;
// whole 16-byte pieces
template <int D, int G>
constexpr int record_floats() { return G * D + (2 * G + 3) / 4 * 4; }
template <int D, int S, int G>
constexpr size_t attn_smem(int nwarp, int ncta) {
  return sizeof(WarpBuffers<D, S>) * nwarp + 1024 + (ncta > 1 ? sizeof(float) * record_floats<D, G>() * ncta : 0);
}

// A cluster of CTAs serves one (sequence, KV head).  Units, dealt to the
// cluster's warps in turn: slices of the incomplete chunk (from the tail),
// then the window's complete chunks and the chosen chunks (tiles of codes).  Each
// warp folds its units with a running maximum per head, the CTA its warps, and
// the cluster its CTAs through distributed shared memory: one launch, no
// workspace, a fixed order of adding.  A warp has one buffer for keys and one for
// values; the next unit's keys are asked for when this one's scores are done, its
// values when this one's sums are.
// Bound by memory where there are many sequences: 64 of 16K, K = 32, W = 512, 32 heads
// over 8, int8: 57.9 us, 5.8 TB/s; 256: 199 us, 6.8 TB/s; 16: 18.9 us, 4.4 TB/s, of
// which the launch, three dependent loads, the first tile's way and the folds are
// about 6.  One sequence, K = 16: 6.6 us, half of it those.
template <typename T, typename C, int D, int S, int G>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) attn_codes_kernel(
    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, Shape s,
    const T* q, CacheView cv, DecView dv, const int32_t* idx, const float* s_sel, T* out, int ncta, DevCtx ctx) {
  using Ops = typename OpsOf<T, C, D, S, G>::type;
  using Slice = TailSlice<T, Ops, D>;
  constexpr int R = Ops::R, N8 = D / 8, KEYS = Slice::KEYS;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[kMaxWarps][2];
  __shared__ int u_tile[kMaxUnits], u_slot[kMaxUnits], n_units;
  __shared__ float red_m[kMaxWarps][G], red_d[kMaxWarps][G];
  unsigned char* smem = align_1k(smem_raw);
  const int nwarp = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, c4 = lane & 3;
  const int rank = blockIdx.x % ncta, g = (int)(blockIdx.x / ncta) % s.Hkv, b = (int)(blockIdx.x / ncta) / s.Hkv;
  uint64_t* bar = bars[warp];
  if (lane == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_barrier_init();
    fence_proxy_async_shared();
  }
  const unsigned long long zero = grid_begin();
  behind(zero, cv), behind(zero, dv), behind(zero, q), behind(zero, idx), behind(zero, s_sel);
  if (lane == 0) fence_proxy_async_all();  // what earlier kernels stored is read by tile copies
  int e0 = -1, e1 = -1;  // the list (warp 0), asked for beside the length
  if (warp == 0) {
    const int32_t* ir = idx + ((long long)b * s.Hkv + g) * s.K;
    if (lane < s.K) e0 = __ldg(ir + lane);
    if (lane + 32 < s.K) e1 = __ldg(ir + lane + 32);
  }
  const int L = dv_len(dv, s, b);
  if (L < 1 || L > s.N) {  // the whole cluster: reported, nothing written
    if (rank == 0 && threadIdx.x == 0) raise_status(ctx, kStatusBadIndex);
    return;
  }
  if (ncta > 1) cluster_arrive();  // waited for before the first CTA's memory is used
  const int cur = (L - 1) / S, wc0 = max(0, cur - s.nw + 1);
  const int n_full = L / S - wc0, part = L % S, n_tail = (part + KEYS - 1) / KEYS;
  if (warp == 0) {
    // the live units: window chunks, then accepted list entries (the list form, common.cuh)
    bool bad;
    accept_list_warp(e0, e1, s.K, wc0, bad);
    if (bad && lane == 0 && rank == 0) raise_status(ctx, kStatusBadIndex);
    const int c[3] = {lane < n_full ? wc0 + lane : -1, e0, e1};
    int tile[3], n = 0;
#pragma unroll
    for (int x = 0; x < 3; ++x) tile[x] = c[x] >= 0 ? dv_tile(dv, s, b, g, c[x], ctx, rank == 0) : -1;
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const unsigned live = __ballot_sync(0xffffffffu, tile[x] >= 0);
      if (tile[x] >= 0) {
        const int at = n + __popc(live & ((1u << lane) - 1u));
        u_tile[at] = tile[x];
        u_slot[at] = x == 0 ? -1 : lane + 32 * (x - 1);
      }
      n += __popc(live);
    }
    if (lane == 0) n_units = n;
  }
  __syncthreads();

  WarpBuffers<D, S>& buf = reinterpret_cast<WarpBuffers<D, S>*>(smem)[warp];
  const int step = ncta * nwarp, end = n_units + n_tail;
  int i = rank * nwarp + warp;
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
  const T* q0 = q + ((long long)b * s.Hq + g * G) * D;
  const TileOffsets<D> at(gq, c4);
  typename Ops::Query qr;
  {
    RawRow<T, D> raw;
    raw.load(Ops::row_head(gq) < G ? q0 + Ops::row_head(gq) * D : (const T*)nullptr, c4);
    Ops::template make_query<T>(raw, gq, c4, qr);
  }

  float acc[R][N8], M[R], den[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    M[r] = -INFINITY;
    den[r] = 0.f;
#pragma unroll
    for (int x = 0; x < N8; ++x) acc[r][x] = 0.f;
  }
  // weights of a unit against the running maximum: fo for what is there, fu for the unit
  auto fold = [&](int r, float lam, float mass, float& fo, float& fu) {
    const float Mn = max_of(M[r], lam);
    fo = exp_neg(M[r] - Mn);
    fu = exp_neg(lam - Mn);
    den[r] = den[r] * fo + fu * mass;
    M[r] = Mn;
  };

  // Of the warp's next 24 units: lane x holds the scales of unit x, lane (gq, c4)
  // the scores of units gq, gq + 8, gq + 16 for its heads.
  float my_ks, my_vs, my_s[R][3];
  auto look_ahead = [&](int i0) {
    my_ks = my_vs = 0.f;
    if (i0 + lane * step < end) {
      const int tile = u_tile[i0 + lane * step - n_tail];
      my_ks = __ldg(cv.k_scale + tile);
      my_vs = __ldg(cv.v_scale + tile);
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const int j = i0 + (gq + 8 * x) * step;
      const int slot = j < end ? u_slot[j - n_tail] : -1;
#pragma unroll
      for (int r = 0; r < R; ++r)
        my_s[r][x] = slot >= 0 && Ops::head(r, c4) < G
                         ? __ldg(s_sel + ((long long)b * s.Hq + g * G + Ops::head(r, c4)) * s.K + slot)
                         : 0.f;
    }
  };
  look_ahead(first);

  for (; i < n_tail; i += step) {
    // the incomplete chunk's keys from KEYS i on, as they are in the tail
    const long long off = tail_off(s, b, g, cur) + KEYS * i * D;
    const T* kt = (const T*)cv.k_tail + off;
    const T* vt = (const T*)cv.v_tail + off;
    const int nk = min(KEYS, part - KEYS * i);
    float sc[R][KEYS / 8];  // keys gq (and gq + 8)
    Slice slice;
    slice.load(kt, vt, q0, nk, G, gq, c4);
    slice.scores(sc);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = -INFINITY, mass = 0.f;
#pragma unroll
      for (int x = 0; x < KEYS / 8; ++x) {
        sc[r][x] = gq + 8 * x < nk ? sc[r][x] * s.scale : -INFINITY;
        top = fmaxf(top, sc[r][x]);
      }
      top = column_max(top);
      const float m = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int x = 0; x < KEYS / 8; ++x) {
        sc[r][x] = exp_neg(sc[r][x] - m);
        mass += sc[r][x];
      }
      float fo, fu;
      fold(r, top, column_sum(mass), fo, fu);
#pragma unroll
      for (int x = 0; x < KEYS / 8; ++x) sc[r][x] *= fu;
#pragma unroll
      for (int x = 0; x < N8; ++x) acc[r][x] *= fo;
    }
    slice.add_values(sc, acc);
  }

  int n_done = 0;
  for (i = first; i < end; i += step, ++n_done) {
    if (n_done == 24) {
      look_ahead(i);
      n_done = 0;
    }
    const int u = i - n_tail, next = i + step < end ? u_tile[u + step] : -1;
    const bool chosen = u_slot[u] >= 0;
    const float ks = __shfl_sync(0xffffffffu, my_ks, n_done), vs = __shfl_sync(0xffffffffu, my_vs, n_done);
    float sc[R][S / 8], o[R][N8], fo[R], fu[R], ls[R];
    alive = mbar_wait(&bar[0], phase[0], ctx);
    if (!__all_sync(0xffffffffu, alive)) break;
    flying[0] = false;
    phase[0] ^= 1u;
    Ops::scores(tile_of<D, S>(buf.a), at, qr, sc);
    __syncwarp();  // every lane has read the keys: their buffer takes the next unit's
    if (next >= 0) {
      if (lane == 0) fetch_tile<D, S>(buf.a, &kmap, next, &bar[0], ctx);
      flying[0] = true;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top, l;
      weigh<Ops>(sc[r], s.scale * ks * qr.up[r], top, l);
      ls[r] = chosen ? l : Ops::kOne;
      // a chosen chunk weighs e^{s^} whatever its l; a window chunk e^{top} l
      const float mine = n_done < 8 ? my_s[r][0] : n_done < 16 ? my_s[r][1] : my_s[r][2];
      const float shat = __shfl_sync(0xffffffffu, mine, 4 * (n_done & 7) + c4);
      fold(r, chosen ? shat : top, chosen ? 1.f : l * (1.f / Ops::kOne), fo[r], fu[r]);
    }
    alive = mbar_wait(&bar[1], phase[1], ctx);
    if (!__all_sync(0xffffffffu, alive)) break;
    flying[1] = false;
    phase[1] ^= 1u;
    Ops::values(tile_of<D, S>(buf.b), at, gq, sc, o, [] {});
    __syncwarp();
    if (next >= 0) {
      if (lane == 0) fetch_tile<D, S>(buf.b, &vmap, next, &bar[1], ctx);
      flying[1] = true;
    }
    const float lifted = lift(vs, o);
#pragma unroll
    for (int r = 0; r < R; ++r) fu[r] *= __fdividef(lifted, ls[r]);
    bool same = true;  // no column's maximum moved
#pragma unroll
    for (int r = 0; r < R; ++r) same = same && fo[r] == 1.f;
    if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int x = 0; x < N8; ++x) acc[r][x] *= fo[r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int x = 0; x < N8; ++x) acc[r][x] = fmaf(o[r][x], fu[r], acc[r][x]);
  }
  if (!__all_sync(0xffffffffu, alive) && lane == 0 && ctx.inject != 1) {
    // a wait ran out: let the copies in flight land before the buffers change hands
    if (flying[0]) mbar_wait(&bar[0], phase[0], ctx);
    if (flying[1]) mbar_wait(&bar[1], phase[1], ctx);
  }
  __syncthreads();  // every warp's copies have landed and been read: the buffers now hold the records

  float* rec = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int h = Ops::head(r, c4);
    if (h >= G) continue;
#pragma unroll
    for (int x = 0; x < N8; x += 4)
      *reinterpret_cast<float4*>(rec + (warp * G + h) * D + gq * N8 + x) =
          make_float4(acc[r][x], acc[r][x + 1], acc[r][x + 2], acc[r][x + 3]);
    if (gq == 0) {
      red_m[warp][h] = M[r];
      red_d[warp][h] = den[r];
    }
  }
  __syncthreads();
  // the records of a cluster's CTAs, in its first one, behind the warps' buffers
  float* records = reinterpret_cast<float*>(smem + sizeof(WarpBuffers<D, S>) * nwarp);
  float* mine = records + rank * record_floats<D, G>();
  if (ncta > 1) cluster_wait();  // every CTA of the cluster has started
  T* o0 = out + ((long long)b * s.Hq + g * G) * D;
  // four dims of a head at a time
  auto add = [](float4& n, float f, const float4& x) {
    n.x = fmaf(f, x.x, n.x), n.y = fmaf(f, x.y, n.y), n.z = fmaf(f, x.z, n.z), n.w = fmaf(f, x.w, n.w);
  };
  auto write = [&](int x, const float4& n, float d) {
    const float4 y = make_float4(n.x / d, n.y / d, n.z / d, n.w / d);
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(o0 + x) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    else
      *reinterpret_cast<float4*>(o0 + x) = y;
  };
  for (int x = 4 * threadIdx.x; x < G * D; x += 4 * blockDim.x) {
    const int h = x / D;
    float Mx = kLeast, dd = 0.f;
#pragma unroll 4
    for (int w = 0; w < nwarp; ++w) Mx = fmaxf(Mx, red_m[w][h]);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int w = 0; w < nwarp; ++w) {
      const float f = exp_neg(red_m[w][h] - Mx);
      add(num, f, *reinterpret_cast<const float4*>(rec + w * G * D + x));
      dd = fmaf(f, red_d[w][h], dd);
    }
    if (ncta == 1) {
      write(x, num, dd);
    } else {
      store_first(mine + x, num);
      if (x % D == 0) {
        store_first(mine + G * D + 2 * h, Mx);
        store_first(mine + G * D + 2 * h + 1, dd);
      }
    }
  }
  if (ncta == 1) return;
  cluster_arrive();
  cluster_wait();
  if (rank > 0) return;
  for (int x = 4 * threadIdx.x; x < G * D; x += 4 * blockDim.x) {
    const int h = x / D;
    float Mx = kLeast, dd = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kMaxCtas; ++w)
      if (w < ncta) Mx = fmaxf(Mx, records[w * record_floats<D, G>() + G * D + 2 * h]);
#pragma unroll
    for (int w = 0; w < kMaxCtas; ++w) {
      if (w >= ncta) continue;
      const float* r = records + w * record_floats<D, G>();
      const float f = exp_neg(r[G * D + 2 * h] - Mx);
      add(num, f, *reinterpret_cast<const float4*>(r + x));
      dd = fmaf(f, r[G * D + 2 * h + 1], dd);
    }
    write(x, num, dd);
  }
}

template <typename T, typename C, int D, int S, int G>
cudaError_t go_summ(const Shape& s, const CacheView& cv, const DecView& dv, const void* q_lmk, const LmkStrides& ls,
                    const int* from, void* k_sum, float* b_sum, cudaStream_t st, const DevCtx& ctx) {
  if (s.C == 0) return cudaSuccess;
  const size_t smem = sizeof(HalfTiles<D, S>) * kWarps + 1024;
  auto kern = code_summaries_kernel<T, C, D, S, G>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, (int)smem);
  if (e != cudaSuccess) return e;
  CUtensorMap km;
  e = make_tmap_rows128(&km, cv.k_pool, (uint64_t)dv.num_pages * s.Hkv * (S * D / 128), S * D / 256);
  if (e != cudaSuccess) return e;
  // one wave of CTAs, fewer if there are not as many chunks
  const int blocks = (s.B + kSeqs - 1) / kSeqs;
  const long long most = ((long long)(s.B < kSeqs ? s.B : kSeqs) * s.C * s.Hkv + kWarps - 1) / kWarps;
  const long long wave = (device_sm_count() * summary_ctas<T>() + blocks - 1) / blocks;
  return launch_overlapped(kern, dim3((unsigned)(wave < most ? wave : most), blocks), kWarps * 32, smem, 1, st, km, s, cv,
                           dv, (const T*)q_lmk, ls, from, (T*)k_sum, b_sum, ctx);
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
  static_assert(sizeof(float) * G * D <= sizeof(WarpBuffers<D, S>), "a warp's record fits its buffers");
  auto kern = attn_codes_kernel<T, C, D, S, G>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, (int)(attn_smem<D, S, G>(kMaxWarps, 1) > attn_smem<D, S, G>(kMaxWarpsOfMany, kMaxCtas)
                                                               ? attn_smem<D, S, G>(kMaxWarps, 1)
                                                               : attn_smem<D, S, G>(kMaxWarpsOfMany, kMaxCtas)));
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)dv.num_pages * s.Hkv * (S * D / 128);
  e = make_tmap_rows128(&km, cv.k_pool, rows, S * D / 128);
  if (e == cudaSuccess) e = make_tmap_rows128(&vm, cv.v_pool, rows, S * D / 128);
  if (e != cudaSuccess) return e;
  // Warps for each (sequence, KV head): as many as put all of them on the device at
  // once (twelve warps a multiprocessor), so that the memory is busy until they end
  // together; 512 of them with three warps each 57.5 us, with four (two waves) 66.5.
  // Below three a warp's own chain of units is the longer way: 768 with two 102 us,
  // with four 95.  Few of them spread over clusters of CTAs, one multiprocessor
  // each, down to one unit a warp.
  const int sms = device_sm_count(), groups = s.B * s.Hkv;
  const int units = s.K + s.nw - 1 + S / TailSlice<T, typename OpsOf<T, C, D, S, G>::type, D>::KEYS;
  int ncta = sms / groups;
  ncta = ncta < 1 ? 1 : ncta > kMaxCtas ? kMaxCtas : ncta;
  int share = sms * kMaxWarps / groups;
  share = share < 3 ? 4 : share;
  share = share < units ? share : units;
  int nwarp = (share + ncta - 1) / ncta;
  const int most = ncta > 1 ? kMaxWarpsOfMany : kMaxWarps;
  nwarp = nwarp > most ? most : nwarp;
  return launch_overlapped(kern, dim3((unsigned)groups * ncta), nwarp * 32, attn_smem<D, S, G>(nwarp, ncta), ncta,
                           st, km, vm, s, (const T*)q, cv, dv, idx, s_sel, (T*)out, ncta, ctx);
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
