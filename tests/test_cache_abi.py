"""The calls on paged caches without a GPU: every argument that they refuse is refused on the host, before any device
work (the pointers here name no memory)."""
import ctypes

import pytest
import torch

from chunk_wise_sparse_landmark_b200 import hils as H

P = 0x1000
OK = dict(k_pool=P, v_pool=P, k_scale=P, v_scale=P, k_tail=P, v_tail=P, format=H.HILS_KV_I8)
INVALID, UNSUPPORTED = H.HILS_ERR_INVALID_ARG, H.HILS_ERR_UNSUPPORTED


def config(dtype="bf16", **kw):
    base = dict(B=2, N=1024, Hq=8, Hkv=2, d=128, S=64, W=128, K=4) if dtype == "bf16" else dict(
        B=2, N=1024, Hq=8, Hkv=2, d=64, S=32, W=64, K=4)
    return H.make_config(dtype=dtype, **{**base, **kw})


def call(name, cfg, pg=None, cache=None, rows=None, rope=None, **kw):
    lib = H.load()
    pg = H.Paged(P, P, 16 if cfg.chunk == 64 else 64, 100) if pg is None else pg
    c = H.Cache(**OK) if cache is None else cache
    a = [ctypes.byref(cfg), ctypes.byref(pg), ctypes.byref(c)]
    if name == "append":
        return lib.hils_cache_append(*a, ctypes.byref(rows) if rows else None, ctypes.byref(rope) if rope else None, None)
    if name == "summaries":
        return lib.hils_build_summaries_cache(*a, kw.get("q_lmk", P), kw.get("lmk", 0), kw.get("from_lens"), kw.get("k_sum", P), P, None)
    if name == "attn":
        return lib.hils_attn_decode_cache(a[0], kw.get("q", P), a[1], a[2], P, P, kw.get("out", P), kw.get("ws"), 0, None)
    return lib.hils_cache_read(*a, kw.get("k_out", P), kw.get("v_out", P), kw.get("out_rows", 64), None)


CALLS = ("append", "summaries", "attn", "read")


def rows(**kw):
    base = dict(k=P, v=P, q=P, q_out=P + 0x1000, k_row=256, k_head=128, v_row=256, v_head=128, q_row=1024, q_head=128,
                q_out_row=1024, q_out_head=128, row_start=P, positions=None, n_rows=10)
    return H.Rows(**{**base, **kw})


def rope(**kw):
    return H.Rope(**{**dict(cos_table=P, sin_table=P, max_pos=1024, rot_dim=64, interleaved=0), **kw})


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("change", [dict(format=3), dict(format=-1), dict(k_pool=None), dict(v_pool=P + 8), dict(k_scale=None),
                                    dict(v_scale=P + 4), dict(k_tail=None), dict(v_tail=P + 8),
                                    dict(format=H.HILS_KV_NATIVE)])
def test_caches_that_are_refused(name, change):
    """Formats, pools, scales and tails; a native cache with scales and tails."""
    assert call(name, config(), cache=H.Cache(**{**OK, **change}), rows=rows()) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_null_descriptions_are_refused(name):
    lib, cfg = H.load(), config()
    pg, c = H.Paged(P, P, 16, 100), H.Cache(**OK)
    for a in ((None, ctypes.byref(pg), ctypes.byref(c)), (ctypes.byref(cfg), None, ctypes.byref(c)), (ctypes.byref(cfg), ctypes.byref(pg), None)):
        st = {"append": lambda: lib.hils_cache_append(*a, ctypes.byref(rows()), None, None),
              "summaries": lambda: lib.hils_build_summaries_cache(*a, P, 0, None, P, P, None),
              "attn": lambda: lib.hils_attn_decode_cache(a[0], P, a[1], a[2], P, P, P, None, 0, None),
              "read": lambda: lib.hils_cache_read(*a, P, P, 64, None)}[name]()
        assert st == INVALID


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("pg", [H.Paged(None, P, 16, 100), H.Paged(P, P + 2, 16, 100), H.Paged(P, P, 15, 100), H.Paged(P, P, 16, 0)])
def test_page_tables_that_are_refused(name, pg):
    assert call(name, config(), pg=pg, rows=rows()) == INVALID


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw", [dict(dtype="f32", d=32, S=32), dict(dtype="f32", S=16), dict(dtype="bf16", d=64),
                                dict(dtype="bf16", S=32), dict(Hq=32, Hkv=2), dict(K=65), dict(W=64 * 33)])
def test_shapes_that_no_kernel_serves(name, kw):
    cfg = config(**kw)
    assert call(name, cfg, pg=H.Paged(P, P, 64, 100), rows=rows()) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(n_rows=-1), dict(row_start=None), dict(row_start=P + 2), dict(positions=P + 1),
                                dict(k=None), dict(v=P + 8), dict(q=P + 4), dict(q_out=None), dict(k_row=260),
                                dict(v_head=-128), dict(q_head=4), dict(q_out_row=1020), dict(q_out=P, q_out_row=2048)])
def test_rows_that_are_refused(kw):
    assert call("append", config(), rows=rows(**kw)) == INVALID, H.load().hils_last_error()


def test_append_without_rows_is_refused_and_with_none_does_nothing():
    assert call("append", config()) == INVALID
    assert call("append", config(), rows=rows(n_rows=0)) == H.HILS_OK


@pytest.mark.parametrize("kw", [dict(cos_table=None), dict(sin_table=P + 4), dict(max_pos=0), dict(rot_dim=0),
                                dict(rot_dim=24), dict(rot_dim=144), dict(interleaved=2)])
def test_angle_tables_that_are_refused(kw):
    assert call("append", config(), rows=rows(), rope=rope(**kw)) == INVALID


def test_other_arguments_that_are_refused():
    cfg = config()
    for kw in (dict(q_lmk=None), dict(q_lmk=P + 8), dict(lmk=3), dict(lmk=-1), dict(from_lens=P + 2), dict(k_sum=P + 4)):
        assert call("summaries", cfg, **kw) == INVALID, kw
    for kw in (dict(q=None), dict(out=P + 8)):
        assert call("attn", cfg, **kw) == INVALID, kw
    for kw in (dict(k_out=None, v_out=None), dict(k_out=P + 4), dict(out_rows=0), dict(out_rows=-5)):
        assert call("read", cfg, **kw) == INVALID, kw
    native = H.Cache(P, P, None, None, None, None, H.HILS_KV_NATIVE)
    assert call("attn", cfg, cache=native) == INVALID  # a native cache's attention needs its workspace
    assert b"workspace" in H.load().hils_last_error()


def test_outputs_that_lie_on_one_another_are_refused():
    """Rows or heads of q_out with one address, keys and values of a cache or of a read in the same memory."""
    apart = H.Cache(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, H.HILS_KV_I8)
    for kw in (dict(q_out_row=0), dict(q_out_head=0), dict(q_out_head=64), dict(q_out_row=120)):
        assert call("append", config(), cache=apart, rows=rows(**kw)) == INVALID
        assert b"q_out lie on one another" in H.load().hils_last_error(), kw
    for change in (dict(v_pool=P), dict(v_scale=3 * P), dict(v_tail=5 * P)):
        c = H.Cache(*[getattr(apart, f) for f, _ in H.Cache._fields_])
        for f, x in change.items():
            setattr(c, f, x)
        assert call("append", config(), cache=c, rows=rows()) == INVALID
        assert b"share memory" in H.load().hils_last_error(), change
    assert call("read", config(), cache=apart) == INVALID
    assert b"same memory" in H.load().hils_last_error()


@pytest.mark.parametrize("n,Hq,row,head", [(10, 8, 128, 128), (10, 8, 256, 128), (10, 8, 896, 128), (10, 8, 1016, 128),
                                           (10, 8, 128, 1264), (10, 8, 136, 1344), (3, 8, 384, 256), (2, 2, 128, 128),
                                           (2 ** 31 - 1, 8, 128, 2 ** 37), (10, 2, 2 ** 62, 2 ** 62)])
def test_rows_of_q_out_that_lie_between_heads_are_refused(n, Hq, row, head):
    """Strides of at least d that give two rows' heads elements in common."""
    apart = H.Cache(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, H.HILS_KV_I8)
    assert call("append", config(Hq=Hq, Hkv=1), cache=apart, rows=rows(n_rows=n, q_out_row=row, q_out_head=head)) == INVALID
    assert b"q_out lie on one another" in H.load().hils_last_error()


@pytest.mark.parametrize("n,Hq,row,head", [(10, 8, 1024, 128), (10, 8, 128, 1280), (10, 8, 1152, 144), (10, 8, 2048, 136),
                                           (10, 8, 1080, 136), (1, 8, 0, 128), (10, 1, 128, 0), (1, 1, 0, 0),
                                           (2 ** 31 - 1, 8, 128, 2 ** 38), (2, 2, 2 ** 62, 2 ** 61),
                                           (2, 8, 384, 256), (2, 8, 640, 256), (4, 4, 384, 896)])
def test_rows_of_q_out_that_lie_apart_are_taken(n, Hq, row, head):
    """Rows of heads and heads of rows, packed or not, and others that meet nowhere (the call is refused further on: the cache's memory is shared)."""
    c = config(Hq=Hq, Hkv=1)
    shared = H.Cache(P, P, P, P, P, P, H.HILS_KV_I8)
    assert call("append", c, cache=shared, rows=rows(n_rows=n, q_out_row=row, q_out_head=head)) == INVALID
    assert b"share memory" in H.load().hils_last_error()


def test_rope_tables():
    """cos and sin of p base^(-2 i / rot) rounded once to float32, also at far positions."""
    cos, sin = H.rope_tables(200000, 32, base=500000.0, device="cpu")
    assert cos.shape == sin.shape == (200000, 16) and cos.dtype == torch.float32
    a = 199999 * 500000.0 ** (-2 * 3 / 32)
    import math
    assert abs(cos[199999, 3].item() - math.cos(a)) <= 2.0 ** -24 and abs(sin[199999, 3].item() - math.sin(a)) <= 2.0 ** -24
    assert (cos[0] == 1).all() and (sin[0] == 0).all()


def test_the_binding_refuses_tensors_that_do_not_fit():
    """Shapes, types and devices (checked before any call into the library)."""
    pool = torch.zeros((4, 2, 64, 128), dtype=torch.int8)
    scale, tail = torch.zeros((4, 2)), torch.zeros((2, 2, 2, 64, 128), dtype=torch.bfloat16)
    c = H.cache(pool, pool, scale, scale, tail, tail)
    assert c.format == H.HILS_KV_I8
    for bad in ((pool, pool[:3], scale, scale, tail, tail), (pool, pool, scale[:3], scale, tail, tail),
                (pool, pool, scale, scale, tail[:, :1], tail), (pool, pool), (pool.half(), pool.half()),
                (pool.float(), pool.float(), scale, scale)):
        with pytest.raises(AssertionError):
            H.cache(*bad)
    cfg, pg = config(N=128), H.Paged(P, P, 2, 4)
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    for a, kw in (((k.float(), k), {}), ((k[:, :1], k), {}), ((k, k[:2]), {}), ((k, k), dict(q=torch.zeros((3, 8, 128), dtype=torch.bfloat16))),
                  ((k, k), dict(row_start=torch.zeros(2, dtype=torch.int32))), ((k, k), dict(positions=torch.zeros(3))),
                  ((k.transpose(1, 2).contiguous().transpose(1, 2), k), {})):
        with pytest.raises(AssertionError):
            H.hils_cache_append(cfg, pg, c, *a, **kw)
    for other in (config(N=128, Hkv=4), config(N=128, B=3), config("f32", N=128, d=128, S=64, W=128)):
        with pytest.raises(AssertionError):
            H.hils_cache_append(other, pg, c, k, k)
    with pytest.raises(AssertionError):
        H.hils_cache_append(cfg, H.Paged(P, P, 2, 5), c, k, k)  # a table of more pages than the pool has


def test_capacities_and_pools_past_the_kernels_ranges():
    cfg = config(N=2 ** 31 - 10)
    for name in CALLS:
        assert call(name, cfg, pg=H.Paged(P, P, 2 ** 25, 100), rows=rows()) == UNSUPPORTED
        assert call(name, config(), pg=H.Paged(P, P, 16, 2 ** 25), rows=rows()) == UNSUPPORTED  # 2^32 lines of 128 bytes
        assert call(name, config(B=65536), rows=rows()) == UNSUPPORTED
        assert call(name, config(Hq=32768, Hkv=32768), rows=rows()) == UNSUPPORTED


def test_the_module_is_imported_by_a_pytorch_without_cuda():
    """The host's checks work where PyTorch has no CUDA functions (they are taken away here)."""
    import os
    import subprocess
    import sys

    code = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, n)
from chunk_wise_sparse_landmark_b200 import hils as H
cfg = H.make_config(1, 128, 8, 2, 128, 64, 128, 2, torch.bfloat16)
pool = torch.zeros((4, 2, 64, 128), dtype=torch.bfloat16)
k = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
try:
    H.hils_cache_append(cfg, H.Paged(4096, 4096, 2, 4), H.cache(pool, pool), k, k)
except AssertionError as e:
    print("refused:", e)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and "refused: the cache is not on a CUDA device" in r.stdout, r.stderr


class FakeDevices:
    """Two CUDA devices that are only counted: what torch.cuda.device makes current."""

    def __init__(self, monkeypatch):
        self.now = 0
        monkeypatch.setattr(H, "_device", lambda: self.now)
        monkeypatch.setattr(H, "_raw_stream", lambda at: 100 + at)
        monkeypatch.setattr(torch.cuda, "device", self.device)

    def device(self, at):
        import contextlib

        @contextlib.contextmanager
        def current():
            old, self.now = self.now, at
            try:
                yield
            finally:
                self.now = old

        return current()


def test_a_decode_step_is_enqueued_on_the_device_of_its_cache(monkeypatch):
    devices, seen = FakeDevices(monkeypatch), []
    monkeypatch.setattr(H, "hils_score_topk_paged", lambda *a: seen.append(("score", devices.now, a[-1])))
    monkeypatch.setattr(H, "hils_attn_decode_cache",
                        lambda *a: H._launch(dec.cache.at, a[-1], lambda raw: seen.append(("attn", devices.now, raw))))
    dec = H.CacheDecode.__new__(H.CacheDecode)
    dec.cfg, dec.paged, dec.cache = config(), H.Paged(P, P, 16, 100), H.Cache(**OK)
    dec.k_sum = dec.b_sum = dec.idx = dec.s_sel = dec.ws_score = dec.out = dec.ws_attn = None
    for at in (1, 0):
        dec.cache.at = at
        dec.step(None)
        assert seen == [("score", at, None), ("attn", at, 100 + at)] and devices.now == 0
        seen.clear()


def test_a_page_table_on_another_device_than_its_cache_is_refused(monkeypatch):
    """Kernels would read its addresses on the cache's device (devices are only counted here)."""
    FakeDevices(monkeypatch)
    monkeypatch.setattr(H, "_p", lambda t: ctypes.c_void_p(P))
    pg = H.paged(torch.zeros(2, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32), 4)
    assert pg.batch == 2 and pg.at == -1
    pool, scale = torch.zeros((4, 2, 64, 128), dtype=torch.int8), torch.zeros((4, 2))
    tail = torch.zeros((2, 2, 2, 64, 128), dtype=torch.bfloat16)
    c = H.cache(pool, pool, scale, scale, tail, tail)
    c.at, pg.at = 0, 1
    cfg, k = config(N=128), torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    idx, s_sel, q = torch.zeros((2, 2, 4), dtype=torch.int32), torch.zeros((2, 8, 4)), torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    for run in (lambda: H.hils_cache_append(cfg, pg, c, k, k), lambda: H.hils_cache_read(cfg, pg, c, k[None], k[None]),
                lambda: H.hils_build_summaries_cache(cfg, pg, c, q, q, s_sel),
                lambda: H.hils_attn_decode_cache(cfg, q, pg, c, idx, s_sel, q)):
        with pytest.raises(AssertionError, match="page table is on another device"):
            run()
