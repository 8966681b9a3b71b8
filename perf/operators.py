"""Cases of the 8-bit paged cache: appending rows with the position rotation, landmark summaries and decode attention
over the cache, and reading it back.

A cache is a pool of one-chunk pages [pages, Hkv, S, d].  It holds the model's type, or 8-bit codes (int8, e4m3) with
one float32 scale for each page (a block of S tokens) and KV head; a sequence's incomplete chunk is then kept in the
model's type in a tail [B, 2, Hkv, S, d] (chunk c in slot c % 2) and becomes codes when its last token arrives.

`run` computes a case in plain torch operations in 32 bits, or, where `own` is true, by the package's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
MAX_CODE = {"i8": 127.0, "e4m3": 448.0}
CODE_TYPE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -110  # a block whose largest magnitude is below this is held as zeros


# ------------------------------------------------------------------- cases ---

def _case(name, kind, fmt, dtype, B, N, Hq, Hkv, d=128, S=64, W=512, K=32, ragged=False, new=0, rot=128, pairs="halves"):
    return dict(name=name, kind=kind, fmt=fmt, dtype=dtype, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, S=S, W=W, K=K,
                ragged=ragged, new=new, rot=min(rot, d), pairs=pairs)


def listed():
    return [
        # one user's decode step on a 32K context: latency
        _case("attn_1x32k_i8", "attn", "i8", "bf16", 1, 32768, 32, 8, K=16),
        # a full decode batch of long contexts (the decode workload's heads, K and window)
        _case("attn_16x128k_i8", "attn", "i8", "bf16", 16, 131072, 32, 8),
        # a large batch of mixed lengths, eight query heads to a KV head
        _case("attn_96x16k_e4m3", "attn", "e4m3", "bf16", 96, 16384, 64, 8, ragged=True),
        # the float32 path with small heads and chunks
        _case("attn_24x4k_f32_i8", "attn", "i8", "f32", 24, 4096, 16, 4, d=64, S=32, W=128, K=16, ragged=True),
        # summaries of a long prompt that was just written
        _case("summ_1x128k_e4m3", "summ", "e4m3", "bf16", 1, 131072, 32, 8),
        # summaries of a batch of mixed lengths after a restore
        _case("summ_13x8k_i8", "summ", "i8", "bf16", 13, 8200, 16, 8, ragged=True),
        # a prompt into an empty cache of 16-bit pages
        _case("append_1x8k_bf16", "append", "bf16", "bf16", 1, 8192, 32, 8, new=8192),
        # a long prompt into an 8-bit cache, and what its attention will read
        _case("append_1x32k_i8", "append", "i8", "bf16", 1, 32768, 32, 8, new=32768),
        # a serving batch: pieces of prompts beside single decode tokens, partial rotation in neighbouring pairs
        _case("append_21x2k_e4m3", "append", "e4m3", "bf16", 21, 2113, 32, 4, ragged=True, new=640, rot=64, pairs="neighbours"),
        # one token for each sequence into float32 pages
        _case("append_48x1_f32", "append", "f32", "f32", 48, 2048, 16, 4, d=64, S=32, ragged=True, new=1, rot=64),
        # what a layer does in a decode step: append, the summaries of completed chunks, attention
        _case("step_16x32k_i8", "step", "i8", "bf16", 16, 32768, 32, 8, ragged=True, new=1),
        _case("step_1x8k_e4m3", "step", "e4m3", "bf16", 1, 8192, 32, 8, K=16, new=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "summ", "append", "append", "step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"]) if kind in ("attn", "summ") else "bf16"
    fmt = rng.choice(["i8", "e4m3"])
    d, S = (128, 64) if dtype == "bf16" else rng.choice([(64, 32), (64, 64), (128, 32), (128, 64)])
    if kind == "append" and rng.random() < 0.4:  # pages in the model's type
        dtype = rng.choice(["bf16", "f32"])
        fmt, d, S = dtype, *((128, 64) if dtype == "bf16" else rng.choice([(32, 16), (64, 32), (128, 64)]))
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 64)
    most = 1 << 20 if kind in ("attn", "step") else 1 << 17 if kind == "summ" else 1 << 16 if dtype == "bf16" else 1 << 15
    most = min(131072, most // B * 8 // Hkv, most // B * 32 // Hq)
    N = _log(rng, min(300, most), most)
    new = 0
    if kind == "step":
        new = 1
    elif kind == "append":
        new = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, min(N, (1 << 14) * 8 // Hkv * 4 // max(4, Hq // Hkv) // B)))
    c = _case("", kind, fmt, dtype, B, N, Hq, Hkv, d=d, S=S, W=S * _log(rng, 1, 16), K=_log(rng, 1, 64),
              ragged=rng.random() < 0.7, new=min(new, N), rot=rng.choice([d, d // 2]), pairs=rng.choice(["halves", "neighbours"]))
    del c["name"]
    return c


def _lengths(c):
    """(length with the new rows, new rows) of each sequence: part of the case, the same for every seed."""
    rng = random.Random("%(kind)s %(B)d %(N)d %(new)d %(K)d %(ragged)s" % c)
    S, lens, news = c["S"], [], []
    for b in range(c["B"]):
        if c["kind"] in ("attn", "summ"):
            L = rng.randint(1, c["N"]) if c["ragged"] and b else c["N"]
            n = 0
        elif c["new"] == 1:  # one token each; one of a few completes a chunk
            L = rng.randint(1, c["N"]) if c["ragged"] else c["N"]
            if b % 7 == 3 and L >= S:
                L = L // S * S
            n = 1
        elif c["ragged"] and b % 3 == 2:  # a single token beside the pieces
            L, n = rng.randint(1, c["N"]), 1
        else:  # a piece of a prompt; it begins where a chunk begins, as a scheduler cuts prompts
            n = rng.randint(1, c["new"]) if c["ragged"] and b else c["new"]
            L = n + (rng.randint(0, c["N"] - n) // S * S if c["ragged"] else 0)
        lens.append(L)
        news.append(n)
    return lens, news


def _chunk_work(c, L):
    """(chosen chunks, keys of the window, of them in the incomplete chunk) of a decode step at length L."""
    cur, nw = (L - 1) // c["S"], c["W"] // c["S"]
    first = max(0, cur - nw + 1)
    return min(c["K"], first), L - first * c["S"], L % c["S"]


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    ce = e if c["fmt"] in TYPE else 1  # bytes of an element in a page
    lens, news = _lengths(c)
    Hq, Hkv, d, S = c["Hq"], c["Hkv"], c["d"], c["S"]
    by = fl = 0
    if c["kind"] in ("append", "step"):
        T = sum(news)
        by += T * d * (2 * Hq * e + 2 * Hkv * (e + ce)) + T * c["rot"] * 4
        fl += T * (Hq + Hkv) * c["rot"] * 3
        if c["kind"] == "append" and ce == 1:  # read back
            by += sum(lens) * Hkv * d * 2 * (1 + e)
            fl += sum(lens) * Hkv * d * 2
    if c["kind"] in ("attn", "step"):
        for L in lens:
            k, win, part = _chunk_work(c, L)
            by += 2 * Hkv * d * ((k * S + win - part) * ce + part * e) + 2 * Hq * d * e + (k + 16) * 8 * Hkv + k * 4 * (Hq + Hkv)
            fl += 4 * Hq * d * (k * S + win)
    if c["kind"] == "summ":
        for L in lens:
            by += (L // S) * (Hkv * S * d * ce + 4 * Hkv + 2 * Hq * d * e + 4 * Hq)
            fl += (L // S) * 4 * Hq * S * d
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ inputs ---

def _codes(c, pages, g):
    """Codes as blocks of normal keys and values have them, in slices."""
    out = torch.empty((pages, c["Hkv"], c["S"], c["d"]), dtype=CODE_TYPE[c["fmt"]], device=DEV)
    m = MAX_CODE[c["fmt"]]
    step = max(1, (1 << 27) // (c["Hkv"] * c["S"] * c["d"]))
    for p in range(0, pages, step):
        x = torch.randn(out[p:p + step].shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(m / 4).clamp_(-m, m)
        out[p:p + step] = (x.round_() if c["fmt"] == "i8" else x).to(out.dtype)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, N, Hq, Hkv, d, S, K = (c[n] for n in ("B", "N", "Hq", "Hkv", "d", "S", "K"))
    t = TYPE[c["dtype"]]
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(t)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    lens, news = _lengths(c)
    width, C = -(-N // S), N // S
    pages = B * width + 3
    s = dict(c, t=t, pages=pages, lens=ints(lens), longest=max(lens))
    s["table"] = torch.randperm(pages, generator=g, device=DEV)[:B * width].to(torch.int32).reshape(B, width)
    if c["fmt"] in TYPE:
        s["k_pool"], s["v_pool"] = (rand(pages, Hkv, S, d) for _ in range(2))
    else:
        s["k_pool"], s["v_pool"] = _codes(c, pages, g), _codes(c, pages, g)
        s["k_scale"], s["v_scale"] = ((0.8 + 0.4 * torch.rand((pages, Hkv), generator=g, device=DEV)) * (4 / MAX_CODE[c["fmt"]]) for _ in range(2))
        s["k_tail"], s["v_tail"] = (rand(B, 2, Hkv, S, d) for _ in range(2))
    if c["kind"] in ("append", "step"):
        T = sum(news)
        qkv = rand(T, Hq + 2 * Hkv, d)  # the rows of one fused projection
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_out"] = torch.zeros((T, Hq, d), dtype=t, device=DEV)
        s["start"] = ints([sum(news[:b]) for b in range(B + 1)])
        angle = torch.arange(N, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64) * 2 / c["rot"])
        s["cos"], s["sin"] = (f(angle).float().to(DEV) for f in (torch.cos, torch.sin))
    elif c["kind"] == "attn":
        s["q"] = rand(B, Hq, d)
    if c["kind"] in ("attn", "step"):  # lists as the scoring writes them: ascending candidates, then -1
        nw = c["W"] // S
        ncand = ints([max(0, (L - 1) // S - nw + 1) for L in lens])
        width_c = max(K, width)
        r = torch.rand((B, Hkv, width_c), generator=g, device=DEV)
        at = torch.arange(width_c, device=DEV)
        r = torch.where(at < ncand[:, None, None], r, -1.0)
        chosen = r.topk(K, dim=-1)
        idx = torch.where(chosen.values >= 0, chosen.indices, width_c).sort(dim=-1).values
        s["idx"] = torch.where(idx < width_c, idx, -1).to(torch.int32).contiguous()
        s_sel = 4.5 + torch.randn((B, Hq, K), generator=g, device=DEV).abs()
        s["s_sel"] = torch.where(s["idx"].repeat_interleave(Hq // Hkv, dim=1) >= 0, s_sel, -math.inf).contiguous()
        s["out"] = torch.zeros((B, Hq, d), dtype=t, device=DEV)
    if c["kind"] in ("summ", "step"):
        s["q_lmk"] = rand(B, Hq, C, d) if c["kind"] == "summ" else rand(B, Hq, d)
        s["k_sum"] = torch.zeros((B, Hq, C, d), dtype=t, device=DEV)
        s["b_sum"] = torch.zeros((B, Hq, C), device=DEV)
        s["from"] = ints([L - n for L, n in zip(lens, news)]) if c["kind"] == "step" else None
    if c["kind"] == "append" and c["fmt"] not in TYPE:
        s["k_read"], s["v_read"] = (torch.zeros((B, Hkv, s["longest"], d), dtype=t, device=DEV) for _ in range(2))
    if own:  # the descriptions of the cache and of its table that a program makes once
        from chunk_wise_sparse_landmark_b200 import hils as H

        s["cfg"] = H.make_config(B, N, Hq, Hkv, d, S, c["W"], K, t)
        s["paged"] = H.paged(s["lens"], s["table"], pages)
        s["cache"] = H.cache(s["k_pool"], s["v_pool"], s.get("k_scale"), s.get("v_scale"), s.get("k_tail"), s.get("v_tail"))
        if "cos" in s:
            s["rope"] = H.rope(s["cos"], s["sin"], interleaved=c["pairs"] == "neighbours")
    return s


# --------------------------------------------------------- plain operators ---

def _rotate(s, x, pos):
    """The rotation of rows x [T, heads, d] by the angles of their positions."""
    R = s["rot"]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["pairs"] == "neighbours" else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ra, rb], dim=-1).flatten(-2) if s["pairs"] == "neighbours" else torch.cat([ra, rb], dim=-1)
    return torch.cat([y, x[..., R:]], dim=-1).to(s["t"])


def _append(s):
    S, lens, start = s["S"], s["lens"].long(), s["start"].long()
    T, B = s["k"].shape[0], lens.shape[0]
    row = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, row, right=True) - 1
    first = lens - (start[1:] - start[:-1])  # position of each sequence's first new row
    pos = first[seq] + row - start[seq]
    s["q_out"].copy_(_rotate(s, s["q"], pos))
    k, v = _rotate(s, s["k"], pos), s["v"]
    page = s["table"].long()[seq, pos // S]
    if s["fmt"] in TYPE:
        s["k_pool"][page, :, pos % S] = k
        s["v_pool"][page, :, pos % S] = v
        return
    # the chunks that new rows touch: at most (new rows) // S + 2 of each sequence
    base = start // S + 2 * torch.arange(B + 1, device=DEV)
    unit = torch.arange(T // S + 2 * B, device=DEV)
    b = (torch.searchsorted(base, unit, right=True) - 1).clamp(0, B - 1)
    chunk = first[b] // S + unit - base[b]
    full = (chunk + 1) * S <= lens[b]
    live = (chunk * S < lens[b]) & (start[b + 1] > start[b])
    p = chunk[:, None] * S + torch.arange(S, device=DEV)  # the positions of each unit
    new = (p >= first[b][:, None]) & (p < lens[b][:, None]) & live[:, None]
    src = (start[b][:, None] + p - first[b][:, None]).clamp(0, T - 1)
    tails = (s["k_tail"], s["v_tail"])
    blocks = [torch.where(new[:, None, :, None], x[src].transpose(1, 2), tail[b, chunk % 2]) for x, tail in ((k, tails[0]), (v, tails[1]))]
    done = live & full
    at = s["table"].long()[b[done], chunk[done]]
    m = MAX_CODE[s["fmt"]]
    for x, name in zip(blocks, "kv"):
        x = x[done].float()
        top = x.abs().amax(dim=(2, 3))
        fine, zero = torch.isfinite(top), top < TINY
        by = torch.where(fine & ~zero, m / torch.where(zero, 1.0, top), 0.0)
        y = torch.where(fine[..., None, None], x, 0.0) * by[..., None, None]
        pool = s[name + "_pool"]
        if s["fmt"] == "i8":
            pool[at] = y.round().clamp(-m, m).to(pool.dtype)
        else:  # indexing writes single bytes
            pool.view(torch.uint8)[at] = y.clamp(-m, m).to(pool.dtype).view(torch.uint8)
        s[name + "_scale"][at] = torch.where(fine, torch.where(zero, 0.0, top / m), math.nan)
    last = (lens - 1) // S
    u, j = torch.nonzero(new & (chunk >= last[b] - 1)[:, None], as_tuple=True)
    for x, tail in zip(blocks, tails):
        tail[b[u], chunk[u] % 2, :, j] = x[u, :, j]


def _values(s, name, page):
    """The values (float32) of the given pages' heads: page [..., Hkv] -> [..., Hkv, S, d]."""
    head = torch.arange(s["Hkv"], device=DEV)
    pool = s[name + "_pool"]
    if s["fmt"] == "e4m3":
        x = pool.view(torch.uint8)[page, head].view(pool.dtype).float()
    else:
        x = pool[page, head].float()
    return x if s["fmt"] in TYPE else x * s[name + "_scale"][page, head][..., None, None]


def _chunks(s, name, chunk, lens):
    """The values of chunks [B, U, Hkv] of each sequence, the incomplete one from the tail."""
    B = chunk.shape[0]
    at = torch.arange(B, device=DEV)[:, None, None]
    x = _values(s, name, s["table"].long()[at, chunk])
    if s["fmt"] in TYPE:
        return x
    cur = lens // s["S"]  # the incomplete chunk, if lens % S
    tail = s[name + "_tail"][torch.arange(B, device=DEV), cur % 2].float()
    return torch.where((chunk == cur[:, None, None])[..., None, None], tail[:, None], x)


def _attend(s, q):
    B, Hq, Hkv, d, S, K = (s[n] for n in ("B", "Hq", "Hkv", "d", "S", "K"))
    G, nw, lens = Hq // Hkv, s["W"] // S, s["lens"].long()
    cur = (lens - 1) // S
    first = (cur - nw + 1).clamp(min=0)
    win = first[:, None] + torch.arange(nw, device=DEV)  # [B, nw]
    sel = s["idx"].long().transpose(1, 2)  # [B, K, Hkv]
    chunk = torch.cat([sel, win[:, :, None].expand(B, nw, Hkv)], dim=1)
    live = torch.cat([sel >= 0, (win <= cur[:, None])[:, :, None].expand(B, nw, Hkv)], dim=1)
    chunk = torch.where(live, chunk, 0)
    k = _chunks(s, "k", chunk, lens)  # [B, U, Hkv, S, d]
    x = torch.matmul(k, q.float().reshape(B, 1, Hkv, G, d).transpose(-1, -2)) / math.sqrt(d)  # [B, U, Hkv, S, G]
    del k
    p = chunk[..., None] * S + torch.arange(S, device=DEV)
    seen = live[..., None] & (p < lens[:, None, None, None])
    x = torch.where(seen[..., None], x, -math.inf)
    # token weights: e^{s^} softmax(x) in a chosen chunk, e^x in the window; both over their sum
    top = x.amax(dim=3, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    e = torch.exp(x - top)
    z = e.sum(dim=3)  # [B, U, Hkv, G]
    of_sel = s["s_sel"].reshape(B, Hkv, G, K).permute(0, 3, 1, 2)  # [B, K, Hkv, G]
    mass = torch.cat([of_sel, top[:, K:, :, 0] + torch.log(z[:, K:])], dim=1)
    mass = torch.where(live[..., None], mass, -math.inf)
    w = torch.exp(mass - mass.amax(dim=1, keepdim=True))
    w = w / w.sum(dim=1, keepdim=True)
    e = e * torch.where(live[..., None], w / torch.where(z > 0, z, 1.0), 0.0)[:, :, :, None]
    v = torch.where(seen[..., None], _chunks(s, "v", chunk, lens), 0.0)
    o = torch.matmul(e.transpose(-1, -2), v).sum(dim=1)  # [B, Hkv, G, d]
    return o.reshape(B, Hq, d).to(s["t"])


def _summaries(s):
    B, Hq, Hkv, d, S = (s[n] for n in ("B", "Hq", "Hkv", "d", "S"))
    G, lens = Hq // Hkv, s["lens"].long()
    first = torch.zeros_like(lens) if s["from"] is None else s["from"].long() // S
    most = s["N"] // S if s["from"] is None else 1
    chunk = first[:, None] + torch.arange(most, device=DEV)
    live = chunk < (lens // S)[:, None]
    chunk = chunk.clamp(max=s["N"] // S - 1)  # one place for each to write to
    k = _values(s, "k", s["table"].long().gather(1, chunk)[:, :, None].expand(B, most, Hkv))  # [B, c, Hkv, S, d]
    q = s["q_lmk"].float()
    q = q.reshape(B, Hkv, G, -1, d).permute(0, 3, 1, 2, 4)  # [B, c, Hkv, G, d]
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)  # [B, c, Hkv, G, S]
    x = x - x.amax(dim=-1, keepdim=True)
    e = torch.exp(x)
    z = e.sum(dim=-1, keepdim=True)
    p = e / z
    b = (torch.log(z) - (p * x).sum(dim=-1, keepdim=True))[..., 0]
    ks = torch.matmul(p, k).to(s["t"])
    at = chunk[:, None, :].expand(B, Hq, most)
    ks, b = (y.permute(0, 2, 3, 1, *range(4, y.dim())).flatten(1, 2) for y in (ks, b))
    keep = live[:, None, :]
    s["b_sum"].scatter_(2, at, torch.where(keep, b, s["b_sum"].gather(2, at)))
    at = at[..., None].expand(B, Hq, most, d)
    s["k_sum"].scatter_(2, at, torch.where(keep[..., None], ks, s["k_sum"].gather(2, at)))


def _read(s):
    B, Hkv, d, S, R = s["B"], s["Hkv"], s["d"], s["S"], s["longest"]
    lens = s["lens"].long()
    n = -(-R // S)
    chunk = torch.arange(n, device=DEV)[None, :, None].expand(B, n, Hkv)
    keep = (torch.arange(R, device=DEV) < lens[:, None])[:, None, :, None]
    for name in "kv":
        x = _chunks(s, name, chunk, lens).to(s["t"]).transpose(1, 2).reshape(B, Hkv, n * S, d)[:, :, :R]
        s[name + "_read"].copy_(torch.where(keep, x, s[name + "_read"]))


# --------------------------------------------------------------------- run ---

def _run_own(s):
    from chunk_wise_sparse_landmark_b200 import hils as H

    cfg, pg, cache, kind, q = s["cfg"], s["paged"], s["cache"], s["kind"], s.get("q")
    if kind in ("append", "step"):
        H.hils_cache_append(cfg, pg, cache, s["k"], s["v"], q, s["q_out"], s["rope"], s["start"])
        q = s["q_out"]
    if kind in ("summ", "step"):
        H.hils_build_summaries_cache(cfg, pg, cache, s["q_lmk"], s["k_sum"], s["b_sum"], from_lens=s["from"])
    if kind in ("attn", "step"):
        H.hils_attn_decode_cache(cfg, q, pg, cache, s["idx"], s["s_sel"], s["out"])
    if "k_read" in s:
        H.hils_cache_read(cfg, pg, cache, s["k_read"], s["v_read"])


def run(state):
    s, kind = state, state["kind"]
    if own:
        _run_own(s)
    else:
        if kind in ("append", "step"):
            _append(s)
        if kind in ("summ", "step"):
            _summaries(s)
        if kind in ("attn", "step"):
            s["out"].copy_(_attend(s, s["q_out"] if kind == "step" else s["q"]))
        if "k_read" in s:
            _read(s)
    return _outputs(s)


def _outputs(s):
    names = {"attn": ["out"], "summ": ["k_sum", "b_sum"], "step": ["q_out", "k_tail", "v_tail", "k_sum", "b_sum", "out"],
             "append": ["q_out", "k_pool", "v_pool"] if s["fmt"] in TYPE else ["q_out", "k_tail", "v_tail", "k_read", "v_read"]}
    return {n: s[n] for n in names[s["kind"]]}


# ------------------------------------------------------- the same in 64 bits ---

def _exact_rows(s, x, pos):
    """Rotated rows of one sequence in 64 bits, by the complex product."""
    R = s["rot"]
    turn = torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
    y = x.double().clone()
    if s["pairs"] == "neighbours":
        z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) * turn
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def exact(case, seed):
    """One sequence after the other, each sequence's whole context as one array of values."""
    s = prepare(case, seed)
    B, Hq, Hkv, d, S, K = (s[n] for n in ("B", "Hq", "Hkv", "d", "S", "K"))
    G = Hq // Hkv
    lens, news = _lengths(case)
    eight = s["fmt"] not in TYPE
    out = {n: x.double().clone() for n, x in _outputs(s).items()}
    row = 0
    for b in range(B):
        L, n = lens[b], news[b]
        pages = s["table"][b, :-(-L // S)].long()
        need = range(len(pages))
        if s["kind"] in ("attn", "step"):  # the chunks that the step reads
            need = sorted(set(s["idx"][b].flatten().tolist()) - {-1} | set(range(max(0, (L - 1) // S - s["W"] // S + 1), (L - 1) // S + 1)))
        at = torch.tensor(list(need), device=DEV)
        ctx = {}
        for name in "kv":
            pool = s[name + "_pool"]
            x = (pool.view(torch.uint8)[pages[at]].view(pool.dtype) if s["fmt"] == "e4m3" else pool[pages[at]]).double()
            if eight:
                x = x * s[name + "_scale"][pages[at]].double()[..., None, None]
                if L // S in need:
                    x[list(need).index(L // S)] = s[name + "_tail"][b, L // S % 2].double()
            ctx[name] = x
        if n:
            pos = torch.arange(L - n, L, device=DEV)
            mine = slice(row, row + n)
            out["q_out"][mine] = _exact_rows(s, s["q"][mine], pos)
            k_new = _exact_rows(s, s["k"][mine], pos)
            for name, x in (("k", k_new), ("v", s["v"][mine].double())):
                old = s[name + "_tail"][b].double().clone() if eight else None
                for c in range((L - n) // S, (L - 1) // S + 1):
                    lo, hi = max(c * S, L - n), min(c * S + S, L)
                    part = x[lo - L + n:hi - L + n].transpose(0, 1)
                    if not eight:
                        out[name + "_pool"][pages[c], :, lo - c * S:hi - c * S] = part
                        continue
                    block = old[c % 2].clone()
                    block[:, lo - c * S:hi - c * S] = part
                    if c >= (L - 1) // S - 1:
                        out[name + "_tail"][b, c % 2, :, lo - c * S:hi - c * S] = part
                    if hi == c * S + S:  # held in 8 bits from now on
                        m = MAX_CODE[s["fmt"]]
                        block = block.to(s["t"]).double()
                        top = block.abs().amax(dim=(1, 2), keepdim=True)
                        y = block / top * m
                        block = (y.round() if s["fmt"] == "i8" else y.float().to(torch.float8_e4m3fn).double()) * (top / m)
                    if c in need:
                        ctx[name][list(need).index(c)] = block
            row += n
        if "k_read" in out:
            for name in "kv":
                out[name + "_read"][b, :, :L] = ctx[name].transpose(0, 1).reshape(Hkv, -1, d)[:, :L]
        if s["kind"] in ("summ", "step"):
            for c in range((L - n) // S if n else 0, L // S):
                k = ctx["k"][list(need).index(c)] if n else ctx["k"][c]
                q = (s["q_lmk"][b].reshape(Hkv, G, d) if n else s["q_lmk"][b, :, c].reshape(Hkv, G, d)).double()
                p = torch.softmax(torch.einsum("hgd,hsd->hgs", q, k) / math.sqrt(d), dim=-1)
                out["k_sum"][b, :, c] = torch.einsum("hgs,hsd->hgd", p, k).reshape(Hq, d)
                out["b_sum"][b, :, c] = torch.special.entr(p).sum(dim=-1).reshape(Hq)
        if s["kind"] in ("attn", "step"):
            q = (out["q_out"][row - 1].to(s["t"]) if n else s["q"][b]).double().reshape(Hkv, G, d)
            first = max(0, (L - 1) // S - s["W"] // S + 1)
            w0 = list(need).index(first)
            kw, vw = (ctx[n].transpose(0, 1)[:, w0:].reshape(Hkv, -1, d)[:, :L - first * S] for n in "kv")
            x = torch.einsum("hgd,htd->hgt", q, kw) / math.sqrt(d)
            lists = s["idx"][b].long()
            of = torch.searchsorted(at, lists.clamp(min=0)).clamp(max=len(need) - 1)  # [Hkv, K]
            head = torch.arange(Hkv, device=DEV)[:, None]
            kc, vc = (ctx[n][of, head] for n in "kv")  # [Hkv, K, S, d]
            oc = torch.einsum("hgks,hksd->hgkd", torch.softmax(torch.einsum("hgd,hksd->hgks", q, kc) / math.sqrt(d), dim=-1), vc)
            score = s["s_sel"][b].double().reshape(Hkv, G, K)
            score = torch.where(lists[:, None] >= 0, score, -math.inf)
            w = torch.softmax(torch.cat([score, x], dim=-1), dim=-1)
            out["out"][b] = (torch.einsum("hgk,hgkd->hgd", w[..., :K], oc) + torch.einsum("hgt,htd->hgd", w[..., K:], vw)).reshape(Hq, d)
    if s["kind"] == "step":  # a key next to a border of its rounding moves a code, and this by more than 32 bits resolve
        out["b_sum"] = None
    return out
