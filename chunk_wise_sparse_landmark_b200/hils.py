"""Thin Python binding of libhils.so (C ABI in include/hils.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch tensors supply device memory and the current CUDA stream.
The library is loaded from this package's directory; if it is missing the
first call raises (there is no fallback of any kind).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhils.so")

HILS_OK, HILS_ERR_INVALID_ARG, HILS_ERR_UNSUPPORTED, HILS_ERR_CUDA, HILS_ERR_TIMEOUT = range(5)
HILS_F32, HILS_BF16 = 0, 1
(HILS_WS_SCORE_PREFILL, HILS_WS_SCORE_DECODE, HILS_WS_ATTN_DECODE, HILS_WS_PREFILL_HOST, HILS_WS_ATTN_PREFILL,
 HILS_WS_PREFILL_BWD) = range(6)
HILS_KV_NATIVE, HILS_KV_I8, HILS_KV_E4M3 = range(3)
HILS_LMK_CHUNK, HILS_LMK_SEQUENCE, HILS_LMK_SHARED = range(3)

EXPORTS = (
    "hils_build_summaries",
    "hils_build_summaries_shared",
    "hils_score_topk",
    "hils_attn_prefill",
    "hils_attn_decode",
    "hils_attn_decode_noalloc",
    "hils_prefill_host",
    "hils_prefill_bwd",
    "hils_decode_append",
    "hils_build_summaries_paged",
    "hils_score_topk_paged",
    "hils_attn_decode_paged",
    "hils_cache_append",
    "hils_build_summaries_cache",
    "hils_attn_decode_cache",
    "hils_cache_read",
    "hils_host_device_pointer",
    "hils_workspace_bytes",
    "hils_sync_status",
    "hils_last_error",
    "hils_set_wait_budget",
    "hils_set_fault_injection",
    "hils_version",
)


class HilsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"hils status {status}: {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("seq_len", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("chunk", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("query_block", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int32),
    ]


class QCal(ctypes.Structure):
    _fields_ = [
        ("h", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p),
        ("w_up", ctypes.c_void_p),
        ("rank", ctypes.c_int32),
        ("d_model", ctypes.c_int32),
    ]


class Paged(ctypes.Structure):
    """A paged, chunk-aligned decode cache (include/hils.h, hils_paged_t)."""
    _fields_ = [
        ("seq_lens", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
    ]
    batch = at = None  # sequences and CUDA device of the tables, where known (paged())


class Cache(ctypes.Structure):
    """A paged cache of any format (include/hils.h, hils_cache_t)."""
    _fields_ = [
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("k_tail", ctypes.c_void_p),
        ("v_tail", ctypes.c_void_p),
        ("format", ctypes.c_int32),
    ]


class Rows(ctypes.Structure):
    """The new rows of an append (include/hils.h, hils_rows_t)."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("k_row", ctypes.c_int64),
        ("k_head", ctypes.c_int64),
        ("v_row", ctypes.c_int64),
        ("v_head", ctypes.c_int64),
        ("q_row", ctypes.c_int64),
        ("q_head", ctypes.c_int64),
        ("q_out_row", ctypes.c_int64),
        ("q_out_head", ctypes.c_int64),
        ("row_start", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("n_rows", ctypes.c_int32),
    ]


_ROWS = struct.Struct("4P8q2Pi4x")  # the same as bytes, cheaper to make for a call
assert _ROWS.size == ctypes.sizeof(Rows)


class Rope(ctypes.Structure):
    """Angle tables of the rotary position embedding (include/hils.h, hils_rope_t)."""
    _fields_ = [
        ("cos_table", ctypes.c_void_p),
        ("sin_table", ctypes.c_void_p),
        ("max_pos", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
    ]


_lib = None


def load() -> ctypes.CDLL:
    """Load libhils.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m chunk_wise_sparse_landmark_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, C = ctypes.c_void_p, ctypes.POINTER(Config)
        lib.hils_build_summaries.argtypes = [C, P, P, P, P, P]
        lib.hils_build_summaries_shared.argtypes = [C, P, P, P, P, P]
        lib.hils_score_topk.argtypes = [C, P, ctypes.POINTER(QCal), P, P, P, P, P, ctypes.c_size_t, ctypes.c_int32, P]
        lib.hils_attn_prefill.argtypes = [C, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.hils_attn_decode.argtypes = [C, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.hils_attn_decode_noalloc.argtypes = [C, P, P, P, P, P, P, P]
        lib.hils_prefill_host.argtypes = [C, P, P, P, P, ctypes.POINTER(QCal), P, P, ctypes.c_size_t, P]
        lib.hils_prefill_bwd.argtypes = [C, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.hils_host_device_pointer.argtypes = [P, ctypes.POINTER(ctypes.c_void_p)]
        lib.hils_host_device_pointer.restype = ctypes.c_int
        PG = ctypes.POINTER(Paged)
        lib.hils_decode_append.argtypes = [C, PG, P, P, P, P, P, P, P, P]
        lib.hils_build_summaries_paged.argtypes = [C, PG, P, P, P, P, P]
        lib.hils_score_topk_paged.argtypes = [C, P, PG, P, P, P, P, P, ctypes.c_size_t, P]
        lib.hils_attn_decode_paged.argtypes = [C, P, P, P, PG, P, P, P, P, ctypes.c_size_t, P]
        # descriptions go by their addresses (_at), the cheapest form of a call
        lib.hils_cache_append.argtypes = [P, P, P, P, P, P]
        lib.hils_build_summaries_cache.argtypes = [P, P, P, P, ctypes.c_int32, P, P, P, P]
        lib.hils_attn_decode_cache.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.hils_cache_read.argtypes = [P, P, P, P, P, ctypes.c_int32, P]
        lib.hils_workspace_bytes.argtypes = [C, ctypes.c_int32, ctypes.c_int32]
        lib.hils_workspace_bytes.restype = ctypes.c_size_t
        lib.hils_sync_status.argtypes = [P]
        lib.hils_last_error.restype = ctypes.c_char_p
        lib.hils_set_wait_budget.argtypes = [ctypes.c_int64]
        lib.hils_set_wait_budget.restype = None
        lib.hils_set_fault_injection.argtypes = [ctypes.c_int32]
        lib.hils_set_fault_injection.restype = None
        lib.hils_version.restype = ctypes.c_char_p
        for n in ("hils_build_summaries", "hils_build_summaries_shared", "hils_score_topk", "hils_attn_prefill",
                  "hils_attn_decode", "hils_attn_decode_noalloc", "hils_prefill_host", "hils_prefill_bwd",
                  "hils_decode_append", "hils_build_summaries_paged", "hils_score_topk_paged",
                  "hils_attn_decode_paged", "hils_cache_append", "hils_build_summaries_cache",
                  "hils_attn_decode_cache", "hils_cache_read", "hils_sync_status"):
            getattr(lib, n).restype = ctypes.c_int
        _lib = lib
    return _lib


def make_config(B, N, Hq, Hkv, d, S, W, K, dtype, M=0, scale=0.0) -> Config:
    dt = HILS_F32 if dtype in ("f32", torch.float32, HILS_F32) else HILS_BF16
    return Config(B, N, Hq, Hkv, d, S, W, K, M, scale, dt)


def config_of(w) -> Config:
    """Config for an :class:`inputs.Workload`."""
    return make_config(w.B, w.N, w.Hq, w.Hkv, w.d, w.S, w.W, w.K, w.dtype, M=w.M)


def _p(t: torch.Tensor | None):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors"
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st: int):
    if st != HILS_OK:
        raise HilsError(st, load().hils_last_error().decode())


def workspace_bytes(cfg: Config, which: int, qcal_rank: int = 0) -> int:
    n = load().hils_workspace_bytes(ctypes.byref(cfg), which, qcal_rank)
    if n == ctypes.c_size_t(-1).value:
        raise HilsError(HILS_ERR_INVALID_ARG, load().hils_last_error().decode())
    return n


def hils_build_summaries(cfg: Config, k, q_lmk, k_sum, b_sum, stream=None):
    _check(load().hils_build_summaries(ctypes.byref(cfg), _p(k), _p(q_lmk), _p(k_sum), _p(b_sum), _stream(stream)))


def hils_build_summaries_shared(cfg: Config, k, q_shared, k_sum, b_sum, stream=None):
    """Landmark-free summaries: q_shared [Hq, d] is every chunk's landmark query."""
    _check(load().hils_build_summaries_shared(ctypes.byref(cfg), _p(k), _p(q_shared), _p(k_sum), _p(b_sum),
                                              _stream(stream)))


def hils_score_topk(cfg: Config, q, k_sum, b_sum, idx, s_sel, workspace=None, decode=False, qcal=None, stream=None):
    """qcal: None or (h, w_down, w_up) tensors."""
    qc = None
    if qcal is not None:
        h, wd, wu = qcal
        qc = ctypes.byref(QCal(_p(h), _p(wd), _p(wu), wd.shape[0], wd.shape[1]))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hils_score_topk(ctypes.byref(cfg), _p(q), qc, _p(k_sum), _p(b_sum), _p(idx), _p(s_sel),
                                  _p(workspace), ws_bytes, 1 if decode else 0, _stream(stream)))


def hils_attn_prefill(cfg: Config, q, k, v, idx, s_sel, out, workspace=None, stream=None):
    """workspace: None (bf16: the pass without scratch) or a device buffer of
    workspace_bytes(cfg, HILS_WS_ATTN_PREFILL) bytes."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().hils_attn_prefill(ctypes.byref(cfg), _p(q), _p(k), _p(v), _p(idx), _p(s_sel), _p(out),
                                    _p(workspace), ws_bytes, _stream(stream)))


def hils_prefill_bwd(cfg: Config, q, k, v, q_lmk, idx, s_sel, k_sum, dout, dq, dk, dv, dq_lmk, workspace,
                     ds_sel=None, stream=None):
    """Gradients of the prefill (float32 outputs dq, dk, dv, dq_lmk and
    optionally ds_sel), selection held fixed; see include/hils.h."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().hils_prefill_bwd(ctypes.byref(cfg), _p(q), _p(k), _p(v), _p(q_lmk), _p(idx), _p(s_sel), _p(k_sum),
                                   _p(dout), _p(dq), _p(dk), _p(dv), _p(dq_lmk), _p(ds_sel), _p(workspace), ws_bytes,
                                   _stream(stream)))


def paged(seq_lens, block_table, num_pages: int) -> Paged:
    """seq_lens [B] and block_table [B, max_pages] are int32 CUDA tensors."""
    assert seq_lens.dtype == torch.int32 and block_table.dtype == torch.int32
    assert seq_lens.get_device() == block_table.get_device(), "the lengths and the page table are on different devices"
    pg = Paged(_p(seq_lens).value, _p(block_table).value, block_table.shape[1], num_pages)
    pg.tensors = (seq_lens, block_table)  # the description keeps what it points to
    pg.batch, pg.at = min(seq_lens.shape[0], block_table.shape[0]), seq_lens.get_device()
    return pg


def hils_decode_append(cfg: Config, pg: Paged, k_new, v_new, q_lmk_new, k_pool, v_pool, k_sum, b_sum, stream=None):
    _check(load().hils_decode_append(ctypes.byref(cfg), ctypes.byref(pg), _p(k_new), _p(v_new), _p(q_lmk_new),
                                     _p(k_pool), _p(v_pool), _p(k_sum), _p(b_sum), _stream(stream)))


def hils_build_summaries_paged(cfg: Config, pg: Paged, k_pool, q_lmk, k_sum, b_sum, stream=None):
    _check(load().hils_build_summaries_paged(ctypes.byref(cfg), ctypes.byref(pg), _p(k_pool), _p(q_lmk), _p(k_sum),
                                             _p(b_sum), _stream(stream)))


def hils_score_topk_paged(cfg: Config, q, pg: Paged, k_sum, b_sum, idx, s_sel, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().hils_score_topk_paged(ctypes.byref(cfg), _p(q), ctypes.byref(pg), _p(k_sum), _p(b_sum), _p(idx),
                                        _p(s_sel), _p(workspace), ws_bytes, _stream(stream)))


def hils_attn_decode_paged(cfg: Config, q, k_pool, v_pool, pg: Paged, idx, s_sel, out, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().hils_attn_decode_paged(ctypes.byref(cfg), _p(q), _p(k_pool), _p(v_pool), ctypes.byref(pg), _p(idx),
                                         _p(s_sel), _p(out), _p(workspace), ws_bytes, _stream(stream)))


# ------------------------------------------------ caches of any format ---

_at = ctypes.addressof  # of a description


def _dtype(cfg: Config):
    return torch.float32 if cfg.dtype == HILS_F32 else torch.bfloat16


def _t(t: torch.Tensor, shape, dtype, at: int) -> int:
    """Address of a contiguous tensor that must have this shape and type, on CUDA device `at` (-1: CPU)."""
    assert t.size() == shape and t.dtype is dtype and t.get_device() == at and t.is_contiguous(), (
        f"expected a contiguous {dtype} tensor of shape {tuple(shape)} on device {at}, "
        f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, shape, dtype, at: int):
    """Address, row stride and head stride of rows [n, heads, d] whose heads are contiguous."""
    row, head, one = t.stride() if t.ndim == 3 else (0, 0, 0)
    assert one == 1 and t.size() == shape and t.dtype is dtype and t.get_device() == at, (
        f"expected {dtype} rows {tuple(shape)} with contiguous heads on device {at}, "
        f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr(), row, head


# the current stream and device as numbers: what torch.cuda.current_stream() and current_device() are made of, without
# an object for each call (a PyTorch without CUDA has neither, and no tensor that a call would take)
_raw_stream, _device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


def _launch(at: int, stream, fn, *args):
    """fn(*args, stream) on CUDA device `at` (its current stream if None)."""
    raw = _raw_stream(at) if stream is None else stream.cuda_stream
    if _device() != at:
        with torch.cuda.device(at):
            st = fn(*args, raw)
    else:
        st = fn(*args, raw)
    if st:
        _check(st)


def _on(at: int):
    """A context in which CUDA device `at` is the current one."""
    return contextlib.nullcontext() if _device() == at else torch.cuda.device(at)


def cache(k_pool, v_pool, k_scale=None, v_scale=None, k_tail=None, v_tail=None) -> Cache:
    """A paged cache.  Pools [num_pages, Hkv, S, d] of float32 / bfloat16 (native), int8 or
    float8_e4m3fn (8 bits: with float32 scales [num_pages, Hkv] and tails [B, 2, Hkv, S, d])."""
    fmt = {torch.float32: HILS_KV_NATIVE, torch.bfloat16: HILS_KV_NATIVE, torch.int8: HILS_KV_I8,
           torch.float8_e4m3fn: HILS_KV_E4M3}.get(k_pool.dtype)
    assert fmt is not None and k_pool.ndim == 4, "pools are [num_pages, Hkv, S, d] of float32, bfloat16, int8 or float8_e4m3fn"
    at, (pages, hkv, S, d) = k_pool.get_device(), k_pool.shape
    c = Cache(_t(k_pool, k_pool.shape, k_pool.dtype, at), _t(v_pool, k_pool.shape, k_pool.dtype, at), None, None,
              None, None, fmt)
    c.elements = k_pool.dtype
    if fmt != HILS_KV_NATIVE:
        assert k_scale is not None and v_scale is not None and k_tail is not None and v_tail is not None, (
            "an 8-bit cache needs scales and tails")
        c.k_scale, c.v_scale = (_t(x, (pages, hkv), torch.float32, at) for x in (k_scale, v_scale))
        assert k_tail.dtype in (torch.float32, torch.bfloat16)
        tail = (k_tail.shape[0], 2, hkv, S, d)
        c.k_tail, c.v_tail = (_t(x, tail, k_tail.dtype, at) for x in (k_tail, v_tail))
        c.elements = k_tail.dtype
        c.sequences = k_tail.shape[0]
    else:
        assert k_scale is None and v_scale is None and k_tail is None and v_tail is None, (
            "a native cache has no scales and no tails")
        c.sequences = None
    c.at, c.tile, c.pages = at, (hkv, S, d), pages
    c.tensors = (k_pool, v_pool, k_scale, v_scale, k_tail, v_tail)
    return c


def _cache_fits(cfg: Config, pg: Paged, c: Cache):
    assert c.at >= 0, "the cache is not on a CUDA device"
    assert pg.at in (None, c.at), "the page table is on another device than the cache"
    assert c.tile == (cfg.n_kv_heads, cfg.chunk, cfg.head_dim) and c.elements is _dtype(cfg) and (
        pg.num_pages <= c.pages and c.sequences in (None, cfg.batch) and pg.batch in (None, cfg.batch)), "the cache does not fit the configuration or its page table"


def rope(cos, sin, interleaved: bool = False) -> Rope:
    """Angle tables: float32 cos and sin [max_pos, rot_dim / 2]; pairs (x[i], x[i + rot_dim / 2]),
    or (x[2i], x[2i + 1]) if interleaved."""
    assert cos.ndim == 2 and cos.is_cuda
    r = Rope(_t(cos, cos.shape, torch.float32, cos.get_device()), _t(sin, cos.shape, torch.float32, cos.get_device()), cos.shape[0],
             2 * cos.shape[1], int(interleaved))
    r.at = cos.get_device()
    r.tensors = (cos, sin)
    return r


def rope_tables(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos and sin of p base^(-2 i / rot_dim), computed in float64, as float32 [max_pos, rot_dim / 2]."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * base ** (-2 * i / rot_dim)
    return angle.cos().float(), angle.sin().float()


def hils_cache_append(cfg: Config, pg: Paged, cache: Cache, k, v, q=None, q_out=None, rope: Rope | None = None,
                      row_start=None, positions=None, stream=None):
    """Rotate and append: k, v [n, Hkv, d], q and q_out [n, Hq, d] (views with contiguous heads);
    row_start [B + 1] and positions [n] int32."""
    _cache_fits(cfg, pg, cache)
    at, el, n, d = cache.at, cache.elements, k.size(0), cfg.head_dim
    shape = (n, cfg.n_kv_heads, d)
    k, k_row, k_head = _rows(k, shape, el, at)
    v, v_row, v_head = _rows(v, shape, el, at)
    qa = q_row = q_head = oa = o_row = o_head = 0
    if q is not None:
        assert q_out is not None, "q needs q_out"
        shape = (n, cfg.n_q_heads, d)
        qa, q_row, q_head = _rows(q, shape, el, at)
        oa, o_row, o_head = _rows(q_out, shape, el, at)
    start = 0 if row_start is None else _t(row_start, (cfg.batch + 1,), torch.int32, at)
    pos = 0 if positions is None else _t(positions, (n,), torch.int32, at)
    r = _ROWS.pack(k, v, qa, oa, k_row, k_head, v_row, v_head, q_row, q_head, o_row, o_head, start, pos, n)
    if rope is not None:
        assert rope.at == at, "the angle tables are on another device than the cache"
        rope = _at(rope)
    _launch(at, stream, load().hils_cache_append, _at(cfg), _at(pg), _at(cache), r, rope)


def hils_build_summaries_cache(cfg: Config, pg: Paged, cache: Cache, q_lmk, k_sum, b_sum, from_lens=None, stream=None):
    """Summaries over a cache of any format; q_lmk [B, Hq, C, d], one for each sequence
    [B, Hq, d], or one for all [Hq, d]; from_lens [B] int32: only chunks completed since."""
    _cache_fits(cfg, pg, cache)
    at, B, hq, d = cache.at, cfg.batch, cfg.n_q_heads, cfg.head_dim
    C = cfg.seq_len // cfg.chunk
    lmk, shape = {4: (HILS_LMK_CHUNK, (B, hq, C, d)), 3: (HILS_LMK_SEQUENCE, (B, hq, d)),
                  2: (HILS_LMK_SHARED, (hq, d))}[q_lmk.ndim]
    el = cache.elements
    _launch(at, stream, load().hils_build_summaries_cache, _at(cfg), _at(pg), _at(cache),
            _t(q_lmk, shape, el, at), lmk, None if from_lens is None else _t(from_lens, (B,), torch.int32, at),
            _t(k_sum, (B, hq, C, d), el, at), _t(b_sum, (B, hq, C), torch.float32, at))


def hils_attn_decode_cache(cfg: Config, q, pg: Paged, cache: Cache, idx, s_sel, out, workspace=None, stream=None):
    """Decode attention over a cache of any format (workspace: native caches only)."""
    _cache_fits(cfg, pg, cache)
    at, B, hq, K, el = cache.at, cfg.batch, cfg.n_q_heads, cfg.top_k, cache.elements
    ws, ws_bytes = None, 0
    if workspace is not None:
        assert workspace.get_device() == at and workspace.is_contiguous()
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    row = (B, hq, cfg.head_dim)
    _launch(at, stream, load().hils_attn_decode_cache, _at(cfg), _t(q, row, el, at), _at(pg),
            _at(cache), _t(idx, (B, cfg.n_kv_heads, K), torch.int32, at),
            _t(s_sel, (B, hq, K), torch.float32, at), _t(out, row, el, at), ws, ws_bytes)


def hils_cache_read(cfg: Config, pg: Paged, cache: Cache, k_out=None, v_out=None, stream=None):
    """The cache's values as rows k_out, v_out [B, Hkv, rows, d]; rows behind a sequence are left as they were."""
    _cache_fits(cfg, pg, cache)
    some = k_out if k_out is not None else v_out
    assert some is not None and some.ndim == 4, "k_out or v_out [B, Hkv, rows, d] is needed"
    shape = (cfg.batch, cfg.n_kv_heads, some.shape[2], cfg.head_dim)
    k, v = (None if t is None else _t(t, shape, cache.elements, cache.at) for t in (k_out, v_out))
    _launch(cache.at, stream, load().hils_cache_read, _at(cfg), _at(pg), _at(cache), k, v,
            some.shape[2])


def _ph(t: torch.Tensor):
    """Host tensor argument (contiguous CPU memory; pinned for overlapping copies)."""
    assert not t.is_cuda and t.is_contiguous(), "host tensors must be contiguous CPU tensors"
    return ctypes.c_void_p(t.data_ptr())


def hils_prefill_host(cfg: Config, q, k, v, q_lmk, out, workspace, qcal=None, stream=None):
    """The prefill path from host memory (q, k, v, q_lmk, qcal tensors and out on the host)."""
    qc = None
    if qcal is not None:
        h, w_down, w_up = qcal
        qc = ctypes.byref(QCal(_ph(h).value, _ph(w_down).value, _ph(w_up).value, w_down.shape[0], w_down.shape[1]))
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().hils_prefill_host(ctypes.byref(cfg), _ph(q), _ph(k), _ph(v), _ph(q_lmk), qc, _ph(out),
                                    _p(workspace), ws_bytes, _stream(stream)))


def _pc(t):
    """A CUDA tensor, or a device address (int) such as hils_host_device_pointer's."""
    return ctypes.c_void_p(t) if isinstance(t, int) else _p(t)


def hils_attn_decode(cfg: Config, q, k_cache, v_cache, idx, s_sel, out, workspace, stream=None):
    """k_cache / v_cache: CUDA tensors, or device addresses of pinned host memory."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load().hils_attn_decode(ctypes.byref(cfg), _p(q), _pc(k_cache), _pc(v_cache), _p(idx), _p(s_sel), _p(out),
                                   _p(workspace), ws_bytes, _stream(stream)))


def hils_host_device_pointer(t: torch.Tensor) -> int:
    """Device address of a pinned host tensor (for a host-resident decode cache)."""
    assert not t.is_cuda and t.is_pinned() and t.is_contiguous()
    out = ctypes.c_void_p()
    _check(load().hils_host_device_pointer(ctypes.c_void_p(t.data_ptr()), ctypes.byref(out)))
    return out.value


def hils_attn_decode_noalloc(cfg: Config, q, k_cache, v_cache, idx, s_sel, out, stream=None):
    """hils_attn_decode for callers that cannot allocate device memory: the
    partial records go to the library's fixed device scratch (see hils.h)."""
    _check(load().hils_attn_decode_noalloc(ctypes.byref(cfg), _p(q), _p(k_cache), _p(v_cache), _p(idx), _p(s_sel),
                                           _p(out), _stream(stream)))


def hils_sync_status(stream=None):
    _check(load().hils_sync_status(_stream(stream)))


def hils_set_wait_budget(cycles: int):
    load().hils_set_wait_budget(int(cycles))


def hils_set_fault_injection(mode: int):
    load().hils_set_fault_injection(int(mode))


# ------------------------------------------------------------- pipelines ---

def alloc_workspace(nbytes: int, device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)


class Prefill:
    """Buffers and calls for one prefill configuration (all device-resident)."""

    def __init__(self, cfg: Config, device, qcal_rank: int = 0):
        self.cfg = cfg
        B, N, Hq, Hkv, d, S, K = cfg.batch, cfg.seq_len, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.chunk, cfg.top_k
        dt = torch.float32 if cfg.dtype == HILS_F32 else torch.bfloat16
        C = N // S
        self.k_sum = torch.empty((B, Hq, C, d), dtype=dt, device=device)
        self.b_sum = torch.empty((B, Hq, C), dtype=torch.float32, device=device)
        self.idx = torch.empty((B, Hkv, N, K), dtype=torch.int32, device=device)
        self.s_sel = torch.empty((B, Hq, N, K), dtype=torch.float32, device=device)
        self.out = torch.empty((B, Hq, N, d), dtype=dt, device=device)
        self.ws = alloc_workspace(workspace_bytes(cfg, HILS_WS_SCORE_PREFILL, qcal_rank), device)
        self.ws_attn = alloc_workspace(workspace_bytes(cfg, HILS_WS_ATTN_PREFILL), device)

    def run(self, q, k, v, q_lmk, qcal=None, stream=None, shared_lmk=False):
        """shared_lmk: q_lmk is the landmark-free variant's [Hq, d] shared query."""
        if shared_lmk:
            hils_build_summaries_shared(self.cfg, k, q_lmk, self.k_sum, self.b_sum, stream)
        else:
            hils_build_summaries(self.cfg, k, q_lmk, self.k_sum, self.b_sum, stream)
        hils_score_topk(self.cfg, q, self.k_sum, self.b_sum, self.idx, self.s_sel, self.ws, False, qcal, stream)
        hils_attn_prefill(self.cfg, q, k, v, self.idx, self.s_sel, self.out, self.ws_attn, stream)
        return self.out


class Decode:
    """Buffers and calls for one decode configuration; summaries are built by
    :meth:`summarize` (once per cache state) and reused by :meth:`step`."""

    def __init__(self, cfg: Config, device):
        self.cfg = cfg
        B, L, Hq, Hkv, d, S, K = cfg.batch, cfg.seq_len, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.chunk, cfg.top_k
        dt = torch.float32 if cfg.dtype == HILS_F32 else torch.bfloat16
        C = L // S
        self.k_sum = torch.empty((B, Hq, C, d), dtype=dt, device=device)
        self.b_sum = torch.empty((B, Hq, C), dtype=torch.float32, device=device)
        self.idx = torch.empty((B, Hkv, K), dtype=torch.int32, device=device)
        self.s_sel = torch.empty((B, Hq, K), dtype=torch.float32, device=device)
        self.out = torch.empty((B, Hq, d), dtype=dt, device=device)
        self.ws_score = alloc_workspace(workspace_bytes(cfg, HILS_WS_SCORE_DECODE), device)
        self.ws_attn = alloc_workspace(workspace_bytes(cfg, HILS_WS_ATTN_DECODE), device)

    def summarize(self, k_cache, q_lmk, stream=None):
        hils_build_summaries(self.cfg, k_cache, q_lmk, self.k_sum, self.b_sum, stream)

    def step(self, q, k_cache, v_cache, stream=None):
        hils_score_topk(self.cfg, q, self.k_sum, self.b_sum, self.idx, self.s_sel, self.ws_score, True, None, stream)
        hils_attn_decode(self.cfg, q, k_cache, v_cache, self.idx, self.s_sel, self.out, self.ws_attn, stream)
        return self.out


class CacheDecode:
    """Buffers and calls for decoding on a paged cache of any format.

    fmt: "native", "int8" or "e4m3".  The caller owns the page table and the
    lengths (int32 CUDA tensors): block_table [B, >= ceil(seq_len / S)] names
    the pool's pages, seq_lens [B] counts the tokens of each sequence with
    those being appended.  A step of a layer is :meth:`append` (rotation,
    cache, summaries of the chunks it completes) and :meth:`step` (scores,
    selection, attention)."""

    _POOL = {"native": None, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}

    def __init__(self, cfg: Config, seq_lens, block_table, num_pages: int, fmt: str = "int8", rope: Rope | None = None):
        self.cfg, self.rope, self.device = cfg, rope, seq_lens.device
        B, Hq, Hkv, d, S, K = cfg.batch, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.chunk, cfg.top_k
        dt, dev = _dtype(cfg), self.device
        C = cfg.seq_len // S
        assert seq_lens.shape == (B,) and block_table.shape[0] == B
        self.seq_lens, self.block_table = seq_lens, block_table
        self.paged = paged(seq_lens, block_table, num_pages)
        assert fmt in self._POOL, f"fmt is one of {tuple(self._POOL)}"
        el = self._POOL[fmt] or dt
        pools = [torch.zeros((num_pages, Hkv, S, d), dtype=el, device=dev) for _ in range(2)]
        rest = []
        if el is not dt:
            rest = [torch.zeros((num_pages, Hkv), dtype=torch.float32, device=dev) for _ in range(2)]
            rest += [torch.zeros((B, 2, Hkv, S, d), dtype=dt, device=dev) for _ in range(2)]
        self.cache = cache(*pools, *rest)
        self.k_sum = torch.zeros((B, Hq, C, d), dtype=dt, device=dev)
        self.b_sum = torch.zeros((B, Hq, C), dtype=torch.float32, device=dev)
        self.idx = torch.empty((B, Hkv, K), dtype=torch.int32, device=dev)
        self.s_sel = torch.empty((B, Hq, K), dtype=torch.float32, device=dev)
        self.out = torch.empty((B, Hq, d), dtype=dt, device=dev)
        self.ws_score = alloc_workspace(max(16, workspace_bytes(cfg, HILS_WS_SCORE_DECODE)), dev)
        self.ws_attn = None if rest else alloc_workspace(workspace_bytes(cfg, HILS_WS_ATTN_DECODE), dev)

    def append(self, k, v, q_lmk, q=None, q_out=None, row_start=None, from_lens=None, positions=None, stream=None):
        """Rows k, v [n, Hkv, d] (and q -> q_out [n, Hq, d]) of the new tokens, then the summaries of the
        chunks from position from_lens[b] on (all if None) that are complete, by q_lmk
        (:func:`hils_build_summaries_cache`)."""
        hils_cache_append(self.cfg, self.paged, self.cache, k, v, q, q_out, self.rope, row_start, positions, stream)
        hils_build_summaries_cache(self.cfg, self.paged, self.cache, q_lmk, self.k_sum, self.b_sum, from_lens, stream)
        return q_out

    def step(self, q, stream=None):
        """Attention of q [B, Hq, d], each sequence's last token (rotated)."""
        with _on(self.cache.at):  # (the scoring is enqueued on the current device)
            hils_score_topk_paged(self.cfg, q, self.paged, self.k_sum, self.b_sum, self.idx, self.s_sel, self.ws_score,
                                  stream)
        hils_attn_decode_cache(self.cfg, q, self.paged, self.cache, self.idx, self.s_sel, self.out, self.ws_attn, stream)
        return self.out
