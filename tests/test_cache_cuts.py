"""Sequences on an 8-bit paged cache that are cut back, again and again, and appended to: where that may be done
(include/hils.h, hils_cache_t), on the plain model and on the GPU."""
import random

import pytest
import torch

from tests.cache_ref import RefCache


def may_cut(history, S, p):
    """The rule.  history: the (first, end) of the appends so far; p: the length to cut back to, at most the last end."""
    c = p // S
    for r in range(c * S, p):
        last = max((t for t, (a, z) in enumerate(history) if a <= r < z), default=None)
        if last is None or any(z > (c + 2) * S for _, z in history[last:]):
            return False
    return True


def appends(rng, S, cap, steps):
    """Random appends, each at the end or behind a cut that the rule allows: (first, end) pairs."""
    history, L = [], 0
    for _ in range(steps):
        if L and rng.random() < 0.6:
            cuts = [p for p in range(max(0, L - 4 * S), L) if may_cut(history, S, p)]
            L = rng.choice(cuts)
        n = rng.choice([1, 2, S // 2, S - 1, S, 2 * S + 1, rng.randint(1, 3 * S)])
        n = min(n, cap - L)
        if n:
            history.append((L, L + n))
            L += n
    return history


def streams(history, rand):
    """Rows of each append, and the tokens that the sequence consists of after it."""
    now = None
    for a, z in history:
        rows = rand(z - a)
        now = rows if now is None else torch.cat([now[:a], rows])
        yield a, z, rows, now


@pytest.mark.parametrize("seed", range(12))
def test_the_rule_keeps_every_token(seed):
    S, d = 8, 4
    rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    history = appends(rng, S, 80, 30)
    table = torch.arange(10, dtype=torch.int32)[None]
    held = RefCache(1, 1, S, d, torch.float32, table, 10, torch.int8)
    cuts = 0
    for t, (a, z, rows, now) in enumerate(streams(history, lambda n: torch.randn((n, 1, d), generator=gen))):
        cuts += t > 0 and a < history[t - 1][1]
        held.append([z], [z - a], rows, -rows)
        fresh = RefCache(1, 1, S, d, torch.float32, table, 10, torch.int8)
        fresh.append([z], [z], now, -now)
        for x in range(2):
            assert torch.equal(held.values(x, 0, z), fresh.values(x, 0, z)), (t, a, z)
    assert cuts > 5


def test_a_second_cut_below_the_first():
    """Two slots: once a chunk's rows have overwritten those of the chunk two before, that one can be re-entered at its
    first token only, however short the sequence has become."""
    S = 64
    history = [(0, 330), (270, 290)]  # chunk 5 was reached, the sequence now ends in chunk 4
    assert may_cut([(0, 330)], S, 270) and may_cut([(0, 330)], S, 321) and not may_cut([(0, 330)], S, 255)
    assert not any(may_cut(history, S, p) for p in range(193, 256)) and may_cut(history, S, 192)
    assert all(may_cut(history, S, p) for p in range(256, 291))
    assert may_cut(history + [(192, 200)], S, 197) and not may_cut(history + [(192, 200)], S, 191)
    gen = torch.Generator().manual_seed(0)
    table = torch.arange(8, dtype=torch.int32)[None]
    for p, same in ((230, False), (192, True)):  # what the rule is there for
        held, fresh = (RefCache(1, 1, S, 16, torch.float32, table, 8, torch.int8) for _ in range(2))
        for a, z, rows, now in streams(history + [(p, 256)], lambda n: torch.randn((n, 1, 16), generator=gen)):
            held.append([z], [z - a], rows, rows)
        fresh.append([256], [256], now, now)
        assert torch.equal(held.values(0, 0, 256), fresh.values(0, 0, 256)) == same


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("form", ["bf16-i8", "bf16-e4m3", "f32-i8"])
def test_cuts_on_the_gpu(form, seed):
    """Every state is that of a cache which got the sequence's present tokens at once: complete chunks' codes and scales,
    and the rows that are read back."""
    from chunk_wise_sparse_landmark_b200 import hils as H
    from tests.test_gpu_cache import BF, DEV, E4, F32, I8, Case, same

    dtype, code, d, S = {"bf16-i8": (BF, I8, 128, 64), "bf16-e4m3": (BF, E4, 128, 64), "f32-i8": (F32, I8, 64, 32)}[form]
    cap = 10 * S
    c = Case(1, 2, 2, d, S, cap, dtype, code)
    history = [(0, 5 * S + 10), (4 * S + 14, 4 * S + 34), (3 * S, 3 * S + 8), (3 * S + 5, 5 * S), (4 * S + 1, 6 * S + 1)]
    history = history if seed == 0 else appends(random.Random(seed), S, cap, 16)
    for a, z, rows, now in streams(history, lambda n: c.rand(n, 4, d)):
        c.append([z], [z - a], rows[:, :2].contiguous(), rows[:, 2:].contiguous())
        c.check()
        fresh = Case(1, 2, 2, d, S, cap, dtype, code)
        fresh.append([z], [z], now[:, :2].contiguous(), now[:, 2:].contiguous())
        read = []
        for one in (c, fresh):
            read.append([torch.zeros((1, 2, z, d), dtype=dtype, device=DEV) for _ in range(2)])
            H.hils_cache_read(one.cfg, one.paged([z]), one.cache, *read[-1])
            used = one.table[0, :z // S].long().to(DEV)
            read[-1] += [t.view(torch.uint8)[used] if t.dtype is E4 else t[used] for ts in one.dev[:2] for t in ts]
        H.hils_sync_status()
        assert all(same(x, y) for x, y in zip(*read)), (a, z)
