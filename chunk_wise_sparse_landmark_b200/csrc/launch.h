// Internal launchers (C++ linkage, not part of the public ABI).  Shapes have
// been validated by the caller (hils_api.cu); these only enqueue kernels and
// return the launch error.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"
#include "tmap.h"

namespace hils {

struct Shape {
  int B, Hq, Hkv, G, N, d, S, W, nw, K, C, M;
  float scale;
  int dtype;  // 0 f32, 1 bf16
};

// Element offset of the landmark query of (sequence b, query head h, chunk c):
// per-chunk queries use strides (Hq C d, C d, d), a decode step's one query per
// head and sequence (Hq d, d, 0), the landmark-free variant's one shared query
// per head (0, d, 0).
struct LmkStrides {
  long long b, h, c;
  HILS_DI long long of(int bb, int hh, int cc) const { return bb * b + hh * h + cc * c; }
};

// The decode cache as the decode kernels see it.  Default: every sequence has
// length N and its keys and values are contiguous [B, Hkv, N, d].  Paged: a
// pool of one-chunk pages [num_pages, Hkv, S, d]; chunk c of sequence b lives
// in page pages[b * max_pages + c]; sequence b has length seq_lens[b] <= N.
struct DecView {
  const int* seq_lens = nullptr;
  const int* pages = nullptr;
  int max_pages = 0;
  int num_pages = 0;
};
// cache length of sequence b
HILS_DI int dv_len(const DecView& v, const Shape& s, int b) { return v.seq_lens ? __ldg(v.seq_lens + b) : s.N; }
// element offset of the first key of chunk c of (sequence b, KV head g), or -1
// when the page table names a page outside the pool
HILS_DI long long dv_chunk(const DecView& v, const Shape& s, int b, int g, int c) {
  if (!v.pages) return (((long long)b * s.Hkv + g) * s.N + (long long)c * s.S) * s.d;
  if (c < 0 || c >= v.max_pages) return -1;
  const int p = __ldg(v.pages + (long long)b * v.max_pages + c);
  if (p < 0 || p >= v.num_pages) return -1;
  return ((long long)p * s.Hkv + g) * s.S * s.d;
}

// A paged cache of any format (kNative: the shape's type; kI8, kE4M3: one byte
// an element, one scale for each page and KV head, incomplete chunks in the
// tails [B, 2, Hkv, S, d], chunk c in slot c & 1).
enum KvFormat : int { kNative = 0, kI8 = 1, kE4M3 = 2 };
struct CacheView {
  void* k_pool = nullptr;
  void* v_pool = nullptr;
  float* k_scale = nullptr;
  float* v_scale = nullptr;
  void* k_tail = nullptr;
  void* v_tail = nullptr;
  int format = kNative;
};
// the largest magnitude of a code
HILS_DI float max_code(int format) { return format == kI8 ? 127.f : 448.f; }
// element offset of chunk c's tile in a tail
HILS_DI long long tail_off(const Shape& s, int b, int g, int c) {
  return (((long long)b * 2 + (c & 1)) * s.Hkv + g) * s.S * s.d;
}
// the new rows of an append (strides in elements) and the angle tables
struct NewRows {
  const void *k, *v, *q;
  void* q_out;
  long long k_row, k_head, v_row, v_head, q_row, q_head, q_out_row, q_out_head;
  const int* row_start;
  const int* positions;
  int n_rows;
};
struct RopeView {
  const float* cos_t = nullptr;
  const float* sin_t = nullptr;
  int max_pos = 0, rot = 0, interleaved = 0;
};
// Overlapped launches (programmatic dependent launch): a kernel that begins with
// grid_begin() and is launched by launch_overlapped() may be brought onto the
// device while the one before it on the stream still runs, and waits in
// grid_begin() until that one has ended and its writes are visible.  Every thread
// of every CTA calls it before its first access to global memory and before it
// returns.  The returned 0 is added to the pointers that are read afterwards
// (behind()), so that no read of theirs can be moved in front of the wait.
HILS_DI unsigned long long grid_begin() {
  unsigned long long zero;
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;\n\tmov.u64 %0, 0;" : "=l"(zero)::"memory");
  return zero;
}
template <typename P>
HILS_DI void behind(unsigned long long zero, P*& p) {
  p = reinterpret_cast<P*>(reinterpret_cast<unsigned long long>(p) + zero);
}
HILS_DI void behind(unsigned long long zero, CacheView& v) {
  behind(zero, v.k_pool), behind(zero, v.v_pool), behind(zero, v.k_scale), behind(zero, v.v_scale);
  behind(zero, v.k_tail), behind(zero, v.v_tail);
}
HILS_DI void behind(unsigned long long zero, DecView& v) { behind(zero, v.seq_lens), behind(zero, v.pages); }
HILS_DI void behind(unsigned long long zero, NewRows& v) {
  behind(zero, v.k), behind(zero, v.v), behind(zero, v.q), behind(zero, v.q_out), behind(zero, v.row_start);
  behind(zero, v.positions);
}
HILS_DI void behind(unsigned long long zero, RopeView& v) { behind(zero, v.cos_t), behind(zero, v.sin_t); }
// cluster: CTAs of a cluster along x (1: no clusters)
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e != cudaSuccess) cudaGetLastError();  // returned to the caller; later calls must not find it
  return e;
}
cudaError_t launch_cache_append(const Shape& s, const CacheView& cv, const DecView& dv, const NewRows& rows,
                                const RopeView& rope, cudaStream_t st, const DevCtx& ctx);
cudaError_t launch_cache_read(const Shape& s, const CacheView& cv, const DecView& dv, void* k_out, void* v_out,
                              int out_rows, cudaStream_t st, const DevCtx& ctx);
// summaries of chunks [from[b] / S, len[b] / S) over a cache of any format
// (lmk: strides of the landmark queries), and decode attention over an 8-bit one
cudaError_t launch_summaries_cache(const Shape& s, const CacheView& cv, const DecView& dv, const void* q_lmk,
                                   const LmkStrides& lmk, const int* from, void* k_sum, float* b_sum,
                                   cudaStream_t st, const DevCtx& ctx);
cudaError_t launch_attn_codes(const Shape& s, const void* q, const CacheView& cv, const DecView& dv,
                              const int32_t* idx, const float* s_sel, void* out, cudaStream_t st, const DevCtx& ctx);

// K1: landmark summaries (all dtypes); shared_lmk: q_lmk is one query per head
// [Hq, d] shared by every chunk and sequence (the landmark-free variant)
cudaError_t launch_summaries(const Shape& s, const void* k, const void* q_lmk, void* k_sum, float* b_sum,
                             cudaStream_t st, const DevCtx& ctx, bool shared_lmk = false);

// K1 on a paged decode cache (CUDA-core kernel): every complete chunk of each
// sequence (q_lmk [B, Hq, C, d]), or only the chunk the last token completed
// (last_only; q_lmk [B, Hq, d]); k_sum [B, Hq, C, d], b_sum [B, Hq, C]
cudaError_t launch_summaries_paged(const Shape& s, const void* k_pool, const void* q_lmk, void* k_sum, float* b_sum,
                                   const DecView& dv, bool last_only, cudaStream_t st, const DevCtx& ctx);
// the new token's key and value of each sequence into its page (position
// seq_lens[b] - 1); k_new, v_new [B, Hkv, d]
cudaError_t launch_decode_append(const Shape& s, const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                                 const DecView& dv, cudaStream_t st, const DevCtx& ctx);

// fp32 SIMT prefill score + group max + top-K
cudaError_t launch_score_topk_simt(const Shape& s, const void* q, const void* k_sum, const float* b_sum, int32_t* idx,
                                   float* s_sel, cudaStream_t st, const DevCtx& ctx);

// bf16 tensor-core prefill score + group max + top-K (d=128, S=64)
cudaError_t launch_score_topk_tc(const Shape& s, const void* q, const void* k_sum, const float* b_sum, int32_t* idx,
                                 float* s_sel, cudaStream_t st, const DevCtx& ctx);
size_t score_tc_workspace(const Shape& s);

// Q-Cal: q~ = q + W_up W_down h written to q_tilde [B,Hq,N,d] (bf16, d=128)
cudaError_t launch_qcal_tc(const Shape& s, const void* q, const void* h, const void* w_down, const void* w_up,
                           int rank, int d_model, void* q_tilde, cudaStream_t st, const DevCtx& ctx);

// decode score + group max + top-K (all dtypes); workspace: scores
size_t decode_score_workspace(const Shape& s);
cudaError_t launch_score_topk_decode(const Shape& s, const void* q, const void* k_sum, const float* b_sum,
                                     int32_t* idx, float* s_sel, void* ws, cudaStream_t st, const DevCtx& ctx,
                                     const DecView& dv = DecView{});

// fp32 SIMT prefill attention
cudaError_t launch_attn_prefill_simt(const Shape& s, const void* q, const void* k, const void* v, const int32_t* idx,
                                     const float* s_sel, void* out, cudaStream_t st, const DevCtx& ctx);

// bf16 prefill attention (d=128, S=64), one pass that streams each block's
// chunk union (no workspace)
cudaError_t launch_attn_prefill_tc(const Shape& s, const void* q, const void* k, const void* v, const int32_t* idx,
                                   const float* s_sel, void* out, cudaStream_t st, const DevCtx& ctx);
// window attention (tcgen05, two passes over the window chunks, attn_window.cu)
// of positions [t0, t0 + np) of a tile of PT positions (t0 a multiple of 32)
// into a window state of window_state_bytes(s, PT); then the fusion of that
// state with the partial records `part` of the selected chunks into out.  The
// tensor maps of q, k, v are made once per call.
struct WindowMaps {
  CUtensorMap q, k, v;
};
size_t window_state_bytes(const Shape& s, int PT);
cudaError_t make_window_maps(const Shape& s, const void* q, const void* k, const void* v, WindowMaps* m);
cudaError_t launch_attn_window(const Shape& s, const WindowMaps& m, void* wstate, int t0, int np, int PT,
                               cudaStream_t st, const DevCtx& ctx);
cudaError_t launch_attn_fuse(const Shape& s, const int32_t* idx, const float* s_sel, const void* part,
                             const void* wstate, void* out, int t0, int np, int PT, cudaStream_t st);
// bf16 prefill attention, chunk-major selected chunks (tcgen05) + window
// attention and fusion (attn_window.cu), by position tiles; workspace of
// attn_prefill_tc_workspace(s) bytes
size_t attn_prefill_tc_workspace(const Shape& s);
cudaError_t launch_attn_prefill_chunked(const Shape& s, const void* q, const void* k, const void* v,
                                        const int32_t* idx, const float* s_sel, void* out, void* ws,
                                        cudaStream_t st, const DevCtx& ctx);

// decode attention (all dtypes): split-KV partials + merge
size_t decode_attn_workspace(const Shape& s);
cudaError_t launch_attn_decode(const Shape& s, const void* q, const void* k, const void* v, const int32_t* idx,
                               const float* s_sel, void* out, void* ws, cudaStream_t st, const DevCtx& ctx,
                               const DecView& dv = DecView{});

// decode attention with its partial records in a fixed device array (no allocation)
size_t decode_static_scratch_bytes();
cudaError_t launch_attn_decode_static(const Shape& s, const void* q, const void* k, const void* v,
                                      const int32_t* idx, const float* s_sel, void* out, cudaStream_t st,
                                      const DevCtx& ctx);

// backward of the prefill (attention, scores, summaries), CUDA-core kernels;
// workspace of prefill_bwd_workspace(s) bytes; ds_sel may be null
size_t prefill_bwd_workspace(const Shape& s);
cudaError_t launch_prefill_bwd(const Shape& s, const void* q, const void* k, const void* v, const void* q_lmk,
                               const int32_t* idx, const float* s_sel, const void* k_sum, const void* dout, float* dq,
                               float* dk, float* dv, float* dq_lmk, float* ds_sel, void* ws, cudaStream_t st,
                               const DevCtx& ctx);

}  // namespace hils
