"""The 8-bit paged cache at the ends of its ranges: logits so large that a rounding of theirs is a power of e, and so
far below zero that sums of weights must not be taken against a fixed number.

Tolerances are those of test_gpu_cache.py.  Where every softmax of a test gives all its mass to one key, with 100 and
the logits' own errors between it and the next, an error of a logit moves no weight by more than e^-100, so that
the terms with the logits' size drop out (big = wide = 0).
"""
import math

import pytest
import torch

from chunk_wise_sparse_landmark_b200 import hils as H
from tests.cache_ref import attend, rotate, summaries
from tests.test_gpu_cache import BF, DEV, E4, F32, FIXED_Q, I8, Case, expect_bad, out_off, same, weights_off

pytestmark = pytest.mark.gpu

FORMS = [(BF, I8, 1), (BF, I8, 2), (BF, I8, 4), (BF, I8, 8), (BF, E4, 1), (BF, E4, 4), (F32, I8, 2), (F32, E4, 8)]
FORM_IDS = [f"{'bf16' if t is BF else 'f32'}-{'i8' if c is I8 else 'e4m3'}-G{g}" for t, c, g in FORMS]


def one_key_each(c, L, q, k, first=0):
    """Checks, in 64 bits, that in every chunk of the keys k [L, d] one key takes all of each head's mass."""
    logit = (k @ q.T) * c.scale
    wide = (k.abs().sum(dim=1).max() * q.abs().max() * c.scale).item()
    off = 2 * ((c.d + 4) * 2.0 ** -24 + 2.0 ** -22 + FIXED_Q) * wide
    for a in range(first, L - L % c.S, c.S):
        top = logit[a:a + c.S].topk(2, dim=0).values
        assert (top[0] - top[1] >= 100 + 2 * off).all()


def large_keys(c, n, axis, size):
    """n keys along `axis` [d] of signs; in a chunk all of one sign, sizes 0.4 .. 0.9 times `size`, one of them 1 times
    (positive) or 0.3 times it (negative): the logits of a query along the axis have one far above the others."""
    y = size * torch.empty(n).uniform_(0.4, 0.9, generator=c.gen)
    for a in range(0, n, c.S):
        m = min(c.S, n - a)
        at = a + int(torch.randint(m, (1,), generator=c.gen))
        negative = (a // c.S) % 3 == 2
        y[at] = (0.3 if negative else 1.0) * size
        if negative:
            y[a:a + m] *= -1
    return y[:, None] * axis


@pytest.mark.parametrize("times", [1, 100])
@pytest.mark.parametrize("dtype,code,G", FORMS, ids=FORM_IDS)
def test_attention_at_logits_of_ten_thousands_and_more(dtype, code, G, times):
    """Chosen chunks whose logits are 4e4 .. 2e8 or minus those (over a window of zeros), and a window of such
    chunks (one key in it is the largest by far)."""
    B, L, S = 24, 10 * 64 + 5, 64
    c = Case(B, G, 1, 128, S, 11 * S, dtype, code, W=4 * S, K=6)
    axis = torch.randint(0, 2, (128,), generator=c.gen).float() * 2 - 1
    q = ((30 * times * 40 ** torch.rand((B, G, 1), generator=c.gen)) * axis).to(dtype)  # 30 .. 1200, times `times`
    k = torch.zeros((B, L, 128))
    for b in range(B):
        if b % 2 == 0:
            k[b, :7 * S] = large_keys(c, 7 * S, axis, 130.0)
        else:
            k[b] = large_keys(c, L, axis, 65.0)
            k[b, 7 * S + b] = 130.0 * axis  # the window's largest
    k = k.reshape(B * L, 1, 128).to(dtype)
    c.append([L] * B, [L] * B, k, c.rand(B * L, 1, 128))
    idx = torch.tensor([0, 1, 2, 3, 4, 6], dtype=torch.int32).expand(B, 1, 6).contiguous()
    s_sel = 3 + torch.randn((B, G, 6), generator=c.gen)
    out = torch.full((B, G, 128), math.nan, dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged([L] * B), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    off = weights_off(dtype, code, 128, S, 10 * S, 0, 0)
    for b in range(B):
        kk, vv = c.ref.values(0, b, L), c.ref.values(1, b, L)
        one_key_each(c, 7 * S, q[b].double(), kk[0, :7 * S])
        want, mag, low, big, _ = attend(q[b].double(), kk, vv, idx[b].tolist(), s_sel[b].double(), S, c.W, c.scale)
        assert big >= 4e4
        assert out_off(dtype, out[b], want, mag, low, off) <= 0, b


@pytest.mark.parametrize("times", [1, 100])
@pytest.mark.parametrize("dtype,code,G", FORMS, ids=FORM_IDS)
def test_summaries_at_logits_of_ten_thousands_and_more(dtype, code, G, times):
    """Each chunk's summary is its one key, with an entropy of zero."""
    C, S = 60, 64
    c = Case(1, G, 1, 128, S, C * S, dtype, code)
    axis = torch.randint(0, 2, (128,), generator=c.gen).float() * 2 - 1
    ql = ((30 * times * 40 ** torch.rand((1, G, C, 1), generator=c.gen)) * axis).to(dtype)
    k = large_keys(c, C * S, axis, 130.0)[:, None].to(dtype)
    c.append([C * S], [C * S], k, k)
    k_sum, b_sum = torch.zeros((1, G, C, 128), dtype=dtype, device=DEV), torch.zeros((1, G, C), device=DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged([C * S]), c.cache, ql.to(DEV), k_sum, b_sum)
    H.hils_sync_status()
    held = c.ref.values(0, 0, C * S)
    for ch in range(C):
        one_key_each(c, S, ql[0, :, ch].double(), held[0, ch * S:ch * S + S])
    want, ent, mag, low = summaries(held.reshape(1, C, S, 128), ql[0].double(), c.scale)
    assert out_off(dtype, k_sum[0], want, mag, low, weights_off(dtype, code, 128, S, S, 0, 0)) <= 0
    # the one weight's exponent is 0: log and exp of 1, to 2^-20 each
    assert (b_sum[0].double().cpu() - ent).abs().max() <= 2.0 ** -19


@pytest.mark.parametrize("dtype,code,G", [(BF, I8, 4), (BF, E4, 2), (F32, I8, 2), (F32, E4, 8)])
def test_attention_where_every_logit_is_far_below_zero(dtype, code, G):
    """A window of logits below -1e30 (in codes, in the tail, in both): the largest still takes the mass."""
    S = 64
    lens = [S, 2 * S, 20, S + 9, 2 * S]
    B = len(lens)
    c = Case(B, G, 1, 128, S, 8 * S, dtype, code, W=2 * S, K=2)
    axis = torch.randint(0, 2, (128,), generator=c.gen).float() * 2 - 1
    n = sum(lens)
    y = torch.empty(n).uniform_(0.5, 1.0, generator=c.gen)
    for a, L in zip([sum(lens[:b]) for b in range(B)], lens):
        y[a + int(torch.randint(L, (1,), generator=c.gen))] = 0.25
    k = (-2.0 ** 55 * y[:, None, None] * axis).to(dtype)
    q = (2.0 ** 55 * torch.empty((B, G, 1)).uniform_(1, 2, generator=c.gen) * axis).to(dtype)
    c.append(lens, lens, k, c.rand(n, 1, 128))
    idx = torch.full((B, 1, 2), -1, dtype=torch.int32)
    s_sel = torch.full((B, G, 2), -math.inf)
    out = torch.full((B, G, 128), 3.0, dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    for b, L in enumerate(lens):
        want, mag, low, big, _ = attend(q[b].double(), c.ref.values(0, b, L), c.ref.values(1, b, L), idx[b].tolist(),
                                        s_sel[b].double(), S, c.W, c.scale)
        assert big > 1e31 and want.isfinite().all()
        assert out_off(dtype, out[b], want, mag, low, weights_off(dtype, code, 128, S, 2 * S, 0, 0)) <= 0, b


def sequences_taken(start, n_rows):
    """[first, end) of the sequences whose rows the call takes: in [0, n_rows), in order, none before an earlier end."""
    end, taken = 0, []
    for a, z in zip(start, start[1:]):
        fine = 0 <= a <= z <= n_rows
        taken.append((a, z) if fine and a >= end else (0, 0))
        end = max(end, z) if fine else end
    return taken


def row_starts_out_of_order():
    gen = torch.Generator().manual_seed(11)
    many = torch.sort(torch.randint(0, 3000, (701,), generator=gen)).values.tolist()
    for at in torch.randint(0, 701, (40,), generator=gen).tolist():
        many[at] += int(torch.randint(-60, 60, (1,), generator=gen))
    many[100], many[200], many[400], many[500] = 2 ** 31 - 1, -1, 3001, -2 ** 31
    return {"a fall inside": (1000, [0, 1000, 500, 900]), "a fall to the front": (210, [0, 200, 5, 210]),
            "taken behind it": (300, [0, 100, 50, 100, 300]), "past the rows": (60, [0, 99999, 20, 40, 60]),
            "below zero": (40, [-5, 10, 40]), "none taken twice": (256, [0, 128, 64, 192, 128, 256]),
            "nothing taken": (64, [64, 0]), "700 sequences": (3000, many)}


@pytest.mark.parametrize("name", list(row_starts_out_of_order()))
@pytest.mark.parametrize("dtype,d,S,code", [(F32, 64, 32, I8), (BF, 128, 64, None)], ids=["f32-i8", "bf16-native"])
def test_row_starts_out_of_order_lose_no_other_sequence(dtype, d, S, code, name):
    """Each row that two sequences name is the earlier one's; sequences that are skipped are left as they were."""
    n, start = row_starts_out_of_order()[name]
    taken = sequences_taken(start, n)
    B = len(taken)
    c = Case(B, 4, 2, d, S, 1024 if B < 9 else 256, dtype, code, fill=2.0)
    assert all(z - a <= c.cap for a, z in taken) and (B < 9 or 300 < sum(z > a for a, z in taken) < 660)
    angles, rope = c.rope(d, False)
    k, v, q = c.rand(n, 2, d), c.rand(n, 2, d), c.rand(n, 4, d)
    lens = [max(1, z - a) for a, z in taken]
    want = torch.full((n, 4, d), 7.0, dtype=dtype)
    rows = torch.cat([torch.arange(a, z) for a, z in taken])
    pos = torch.cat([torch.arange(z - a) for a, z in taken])
    turn = lambda x: rotate(x, angles[0][pos], angles[1][pos], False)  # noqa: E731
    want[rows] = turn(q[rows])
    q_out = torch.full((n, 4, d), 7.0, dtype=dtype, device=DEV)
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV), v.to(DEV), q.to(DEV), q_out, rope,
                        torch.tensor(start, dtype=torch.int32, device=DEV))
    expect_bad()
    c.ref.append(lens, [z - a for a, z in taken], turn(k[rows]), v[rows])
    c.check()
    assert same(q_out, want)
