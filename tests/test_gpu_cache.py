"""The paged cache of any format on the GPU: appending rotated rows, landmark
summaries, decode attention and reading back, against the plain model of
tests/cache_ref.py.

Tolerances.  What the cache holds (codes, scales, tails, native pages) and the
rotated queries are defined by float32 operations in a given order: equal bits.
For summaries and attention let mag = sum of weight * |value| (from the model):
  * an output element is a weighted sum of at most n held values.  The logits
    are float32 sums of d products: off by at most (d + 4) 2^-24 big, big =
    max sum |q_e k_e| scale (the two scale factors round once each).  A weight is
    off by twice that (its numerator and its sum), and by 2^-20 for exp, log
    and the quotient; sums of S products, then of units: (S + n / S + 16) 2^-24;
  * float32 inputs: queries are held as two halves, within 2^-22 of themselves,
    which a factor of two on the logits' bound covers; weights within 2^-22, or
    2^-40 of the largest of their chunk (low = sum of that largest * |value|);
  * bf16 inputs, half precision (e4m3 codes; int8 codes with eight heads in a
    group): queries exact, or within 2^-39 of their row's largest element, which
    2^-24 big covers; weights within 2^-11, or 2^-40 of the largest of their chunk;
    the result rounds to bf16 (2^-8 of itself);
  * bf16 inputs, int8 digits (up to four heads): queries within 1.02 2^-24 of their
    row's largest element (fixed point, half a step is 1 / 16646144), so a logit
    within that times wide = max |q| sum |k_e| scale; weights within 1.02 2^-16 of
    their chunk's largest (half a step is 1 / 65024).
"""
import math

import numpy as np
import pytest
import torch

from chunk_wise_sparse_landmark_b200 import hils as H
from tests.cache_ref import RefCache, attend, rotate, summaries

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


FIXED_Q, FIXED_P = 1.02 * 2.0 ** -24, 1.02 * 2.0 ** -16


def weights_off(dtype, code, d, S, n, big, wide):
    """Relative error of a weighted sum's terms, and the part of each chunk's largest weight that they resolve."""
    off = 2 * 2 * (d + 4) * 2.0 ** -24 * big + 2.0 ** -20 + (S + n / S + 16) * 2.0 ** -24
    if code is None:
        return off, 0.0
    if dtype is F32:
        return off + 2.0 ** -22, 2.0 ** -40
    return (off + 2 * FIXED_Q * wide + 2.0 ** -11, FIXED_P) if code is I8 else (off + 2.0 ** -11, 2.0 ** -40)


def out_off(dtype, got, want, mag, low, off):
    # the rounding of the result: half a step, which for numbers below 2^-126 is half of bf16's 2^-133 (float32: 2^-149)
    half = (want.abs() * 2.0 ** -8).clamp(min=2.0 ** -134) if dtype is BF else (want.abs() * 2.0 ** -24).clamp(min=2.0 ** -150)
    tol = mag * off[0] + low * off[1] + half
    return ((got.double().cpu() - want).abs() - tol).max().item()


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return torch.equal(bits(a.cpu()), bits(b.cpu()))


class Case:
    """A cache on the GPU beside its model."""

    def __init__(self, B, Hq, Hkv, d, S, cap, dtype, code=None, W=None, K=4, seed=0, fill=0.0, spare=3):
        self.B, self.Hq, self.Hkv, self.d, self.S, self.cap, self.dtype, self.code = B, Hq, Hkv, d, S, cap, dtype, code
        self.W, self.K = W or 2 * S, K
        self.gen = torch.Generator().manual_seed(seed)
        width = -(-cap // S)
        pages = B * width + spare
        self.table = torch.randperm(pages, generator=self.gen)[:B * width].to(torch.int32).reshape(B, width)
        self.ref = RefCache(B, Hkv, S, d, dtype, self.table, pages, code, fill)
        self.cfg = H.make_config(B, cap, Hq, Hkv, d, S, self.W, K, dtype)
        self.dev = [[t.to(DEV) for t in ts] for ts in (self.ref.pool, self.ref.scale, self.ref.tail)]
        (kp, vp), (ks, vs), (kt, vt) = self.dev
        self.cache = H.cache(kp, vp, ks, vs, kt, vt) if code else H.cache(kp, vp)
        self.table_dev, self.pages = self.table.to(DEV), pages
        self.scale = 1.0 / math.sqrt(d)

    def paged(self, lens):
        return H.paged(torch.tensor(lens, dtype=torch.int32, device=DEV), self.table_dev, self.pages)

    def rand(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.gen) * std).to(self.dtype)

    def rope(self, rot, interleaved, max_pos=None):
        cos, sin = H.rope_tables(max_pos or self.cap, rot, device="cpu")
        return (cos, sin), H.rope(cos.to(DEV), sin.to(DEV), interleaved)

    def append(self, lens, news, k, v, q=None, rope=None, angles=None, interleaved=False, positions=None):
        """One call on the GPU and in the model; checks the rotated queries."""
        start = torch.tensor([sum(news[:b]) for b in range(self.B + 1)], dtype=torch.int32, device=DEV)
        pos = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, news)]) if positions is None else positions
        kr = rotate(k, angles[0][pos], angles[1][pos], interleaved) if rope is not None else k
        q_dev = q_out = None
        if q is not None:
            q_dev, q_out = q.to(DEV), torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
        H.hils_cache_append(self.cfg, self.paged(lens), self.cache, k.to(DEV), v.to(DEV), q_dev, q_out, rope, start,
                            None if positions is None else positions.to(torch.int32).to(DEV))
        self.ref.append(lens, news, kr, v)
        if q is not None:
            want = rotate(q, angles[0][pos], angles[1][pos], interleaved) if rope is not None else q
            assert same(q_out, want)

    def check(self):
        H.hils_sync_status()
        for name, got, want in zip(("pool", "scale", "tail"), self.dev, (self.ref.pool, self.ref.scale, self.ref.tail)):
            if self.code is None and name != "pool":
                continue
            for x in range(2):
                assert same(got[x], want[x]), (name, "kv"[x])

    def fill(self, lens):
        """A context of the given lengths in one call."""
        n = sum(lens)
        self.append(lens, lens, self.rand(n, self.Hkv, self.d), self.rand(n, self.Hkv, self.d))

    def lists(self, lens, seed=1):
        """Random lists as the scoring writes them, and scores."""
        rng = np.random.default_rng(seed)
        idx = np.full((self.B, self.Hkv, self.K), -1, dtype=np.int32)
        s_sel = np.full((self.B, self.Hq, self.K), -np.inf, dtype=np.float32)
        for b, L in enumerate(lens):
            cand = max(0, (L - 1) // self.S - self.W // self.S + 1)
            for g in range(self.Hkv):
                pick = np.sort(rng.permutation(cand)[:self.K])
                idx[b, g, :len(pick)] = pick
                G = self.Hq // self.Hkv
                s_sel[b, g * G:(g + 1) * G, :len(pick)] = 3 + rng.standard_normal((G, len(pick)))
        return torch.from_numpy(idx), torch.from_numpy(s_sel)

    def check_attention(self, lens, q, idx, s_sel, out, accepted=None):
        for b, L in enumerate(lens):
            k, v = self.ref.values(0, b, L), self.ref.values(1, b, L)
            want, mag, low, big, wide = attend(q[b].double(), k, v, (idx if accepted is None else accepted)[b].tolist(),
                                    s_sel[b].double(), self.S, self.W, self.scale)
            n = self.K * self.S + self.W
            rel = weights_off(self.dtype, self.code, self.d, self.S, n, big, wide)
            assert out_off(self.dtype, out[b], want, mag, low, rel) <= 0, (b, L)


SHAPES = [(BF, 128, 64), (F32, 64, 32), (F32, 128, 64), (F32, 64, 64), (F32, 128, 32)]
NATIVE = [(BF, 128, 64), (F32, 32, 16), (F32, 64, 32), (F32, 128, 64), (F32, 32, 32), (F32, 64, 16), (F32, 128, 16)]
FORMATS = [(s, c) for c in (I8, E4) for s in SHAPES] + [(s, None) for s in NATIVE]
IDS = [f"{'bf16' if s[0] is BF else 'f32'}-d{s[1]}-S{s[2]}-{'native' if c is None else 'i8' if c is I8 else 'e4m3'}"
       for s, c in FORMATS]
CODED = [(s, c) for c in (I8, E4) for s in SHAPES]
CODED_IDS = IDS[:len(CODED)]


# ------------------------------------------------------------------ append ---

@pytest.mark.parametrize("shape,code", FORMATS, ids=IDS)
def test_append_holds_what_the_model_holds(shape, code):
    """Calls of several sequences: pieces that begin inside a chunk, end inside one, end on a border, cross several
    chunks (both tail slots written and the slot that the first chunk is read from), single tokens, and none."""
    dtype, d, S = shape
    c = Case(4, 4, 2, d, S, 9 * S + 5, dtype, code, fill=2.0)
    angles, rope = c.rope(d, False)
    lens = [0, 0, 0, 0]
    for news in ([S + 3, 1, 2 * S, 0], [S - 3, S - 1, 0, 1], [2 * S + 1, 1, S // 2, S + 1], [1, 3 * S, S // 2, 1],
                 [1, 4 * S, 4 * S + S // 2, 2 * S - 3], [1, 1, 1, 1]):
        lens = [L + n for L, n in zip(lens, news)]
        n = sum(news)
        c.append(lens, news, c.rand(n, 2, d), c.rand(n, 2, d), c.rand(n, 4, d), rope, angles)
        c.check()


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("code", [None, I8], ids=["native", "i8"])
def test_rotation_of_part_of_a_head_and_given_positions(rot, interleaved, code):
    c = Case(2, 8, 1, 128, 64, 300, BF, code)
    angles, rope = c.rope(rot, interleaved, max_pos=5000)
    lens = news = [130, 65]
    pos = torch.randperm(5000, generator=c.gen)[:195]
    c.append(lens, news, c.rand(195, 1, 128), c.rand(195, 1, 128), c.rand(195, 8, 128), rope, angles, interleaved, pos)
    c.check()
    n = [1, 1]  # and two single tokens at the tables' ends
    c.append([131, 66], n, c.rand(2, 1, 128), c.rand(2, 1, 128), c.rand(2, 8, 128), rope, angles, interleaved,
             torch.tensor([0, 4999]))
    c.check()


def test_rotation_against_64_bits():
    """Two products and a sum in float32 (three roundings of at most |a| + |c|), then bf16."""
    c = Case(1, 4, 1, 128, 64, 4096, BF)
    (cos, sin), rope = c.rope(128, False)
    q = c.rand(4096, 4, 128)
    kv = c.rand(4096, 1, 128).to(DEV)
    q_out = torch.empty_like(q, device=DEV)
    H.hils_cache_append(c.cfg, c.paged([4096]), c.cache, kv, kv, q.to(DEV), q_out, rope,
                        torch.tensor([0, 4096], dtype=torch.int32, device=DEV))
    a, b = q[..., :64].double(), q[..., 64:].double()
    co, si = cos.double()[:, None], sin.double()[:, None]
    want = torch.cat([a * co - b * si, b * co + a * si], -1)
    size = torch.cat([a.abs() + b.abs()] * 2, -1)
    assert ((q_out.cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2 * 2.0 ** -24).all()


@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
def test_held_values_are_within_half_a_step(code):
    """int8: half a step is A / 254; e4m3: 2^-4 of the value, or half the smallest step, 2^-10 A / 448; both with the
    float32 roundings of 1 / M, 1 / A and four products (6 * 2^-24 of A)."""
    c = Case(1, 1, 1, 128, 64, 640, BF, code)
    k = c.rand(640, 1, 128) * torch.logspace(-6, 6, 640)[:, None, None].to(BF)
    c.append([640], [640], k, k)
    c.check()
    x = k[:, 0].double().reshape(10, 64, 128)
    A = x.abs().amax(dim=(1, 2), keepdim=True)
    got = c.ref.values(0, 0, 640)[0].reshape(10, 64, 128)
    tol = A / 254 if code is I8 else torch.maximum(x.abs() * 2.0 ** -4, A * (2.0 ** -10 / 448))
    assert ((got - x).abs() <= tol + 6 * 2.0 ** -24 * A).all()


@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_blocks_of_zeros_tiny_huge_and_non_finite_values(dtype, code):
    c = Case(1, 1, 1, 128, 64, 64 * 8, dtype, code)
    k = c.rand(512, 1, 128)
    k[0:64] = 0
    k[64:128] *= 2.0 ** -125  # below the smallest scale that divides
    k[128:192] *= 2.0 ** -100
    k[192:256] *= 2.0 ** 125
    k[300, 0, 7] = math.inf
    k[330, 0, 9] = math.nan
    k[400, 0, 3] = -math.inf
    v = k.flip(0).contiguous()
    c.append([512], [512], k, v)
    H.hils_sync_status()
    for x in range(2):  # NaN scales have no order of bits to compare
        assert same(c.dev[0][x], c.ref.pool[x]) and same(c.dev[2][x], c.ref.tail[x])
        a, b = c.dev[1][x].cpu(), c.ref.scale[x]
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])
        assert int(a.isnan().sum()) == 3  # one in each of three blocks


def test_what_is_held_does_not_depend_on_the_split():
    for code in (I8, E4):
        whole = Case(1, 2, 2, 128, 64, 700, BF, code)
        k, v = whole.rand(700, 2, 128), whole.rand(700, 2, 128)
        whole.append([700], [700], k, v)
        rng = np.random.default_rng(5)
        for _ in range(3):
            cuts = np.sort(rng.choice(np.arange(1, 700), 12, replace=False)).tolist() + [700]
            parts = Case(1, 2, 2, 128, 64, 700, BF, code)
            at = 0
            for z in cuts:
                parts.append([z], [z - at], k[at:z], v[at:z])
                at = z
            H.hils_sync_status()
            for part in range(2):  # pools and scales
                for x in range(2):
                    assert same(parts.dev[part][x], whole.dev[part][x])
            # the tail's rows of the incomplete chunk
            assert same(parts.dev[2][0][0, 10 & 1, :, :60], whole.dev[2][0][0, 10 & 1, :, :60])


def test_a_sequence_cut_back_and_appended_again():
    """Tokens of the last two chunks are dropped and others appended: as if the dropped ones had never been."""
    c = Case(1, 1, 1, 128, 64, 640, BF, I8)
    k, v = c.rand(400, 1, 128), c.rand(400, 1, 128)
    c.append([300], [300], k[:300], v[:300])
    c.append([330], [30], k[300:330], v[300:330])
    c.append([290], [20], k[330:350], v[330:350])  # back to 270, inside the chunk before the last
    want = Case(1, 1, 1, 128, 64, 640, BF, I8)
    kk, vv = torch.cat([k[:270], k[330:350]]), torch.cat([v[:270], v[330:350]])
    want.append([290], [290], kk, vv)
    c.append([330], [40], k[350:390], v[350:390])
    want.append([330], [40], k[350:390], v[350:390])
    H.hils_sync_status()
    for b in range(5):  # complete chunks
        page, page_w = int(c.table[0, b]), int(want.table[0, b])
        assert same(c.dev[0][0][page], want.dev[0][0][page_w]) and same(c.dev[1][1][page], want.dev[1][1][page_w])


def test_views_of_one_projection_head_major_output_and_in_place_queries():
    c = Case(2, 4, 2, 128, 64, 300, BF, I8)
    (angles, rope), n = c.rope(128, False), 200
    lens = news = [150, 50]
    qkv = c.rand(n, 8, 128)
    dev = qkv.to(DEV)
    start = torch.tensor([0, 150, 200], dtype=torch.int32, device=DEV)
    pos = torch.cat([torch.arange(150), torch.arange(50)])
    out = torch.full((4, n, 128), 5.0, dtype=BF, device=DEV)  # [heads, rows, d]
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, dev[:, 4:6], dev[:, 6:], dev[:, :4], out.transpose(0, 1), rope, start)
    c.ref.append(lens, news, rotate(qkv[:, 4:6], angles[0][pos], angles[1][pos], False), qkv[:, 6:])
    c.check()
    want = rotate(qkv[:, :4], angles[0][pos], angles[1][pos], False)
    assert same(out.transpose(0, 1), want)
    # in place, into the same projection
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, dev[:, 4:6], dev[:, 6:], dev[:, :4], dev[:, :4], rope, start)
    c.check()
    assert same(dev[:, :4], want) and same(dev[:, 4:], qkv[:, 4:])


@pytest.mark.parametrize("dtype,d,S", [(BF, 128, 64), (F32, 64, 32)], ids=["bf16", "f32"])
def test_rows_and_heads_of_stride_zero(dtype, d, S):
    """One head for all heads (keys, queries), one row for all rows (values)."""
    c = Case(2, 4, 2, d, S, 5 * S, dtype, E4)
    (angles, rope), n = c.rope(d, False), 3 * S + 7
    lens = news = [2 * S, S + 7]
    k, v, q = c.rand(n, 1, d), c.rand(1, 2, d), c.rand(n, 1, d)
    pos = torch.cat([torch.arange(x) for x in lens])
    out = torch.zeros((n, 4, d), dtype=dtype, device=DEV)
    start = torch.tensor([0, 2 * S, n], dtype=torch.int32, device=DEV)
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV).expand(n, 2, d), v.to(DEV).expand(n, 2, d),
                        q.to(DEV).expand(n, 4, d), out, rope, start)
    turn = lambda x: rotate(x, angles[0][pos], angles[1][pos], False)
    c.ref.append(lens, news, turn(k.expand(n, 2, d)), v.expand(n, 2, d).contiguous())
    c.check()
    assert same(out, turn(q.expand(n, 4, d)).contiguous())
    with pytest.raises(H.HilsError, match="lie on one another"):
        H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV).expand(n, 2, d), v.to(DEV).expand(n, 2, d),
                            q.to(DEV).expand(n, 4, d), out[:, :1].expand(n, 4, d), rope, start)


def offset(t):
    """A copy on the GPU that begins 16 bytes behind a 512-byte border."""
    n = 16 // t.element_size()
    store = torch.zeros(t.numel() + n, dtype=torch.uint8 if t.dtype is E4 else t.dtype, device=DEV)
    view = store[n:].view(t.dtype).view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 32 == 16
    return view


@pytest.mark.parametrize("shape,code", [((BF, 128, 64), I8), ((BF, 128, 64), E4), ((F32, 64, 32), I8), ((BF, 128, 64), None)],
                         ids=["bf16-i8", "bf16-e4m3", "f32-i8", "native"])
def test_every_tensor_at_16_byte_alignment(shape, code):
    dtype, d, S = shape
    lens = [3 * S + 5, 2 * S]
    n = sum(lens)
    c = Case(2, 4, 2, d, S, 4 * S, dtype, code, W=S, K=2)
    c.dev = [[offset(t) for t in ts] for ts in c.dev]
    (kp, vp), (ks, vs), (kt, vt) = c.dev
    c.cache = H.cache(kp, vp, ks, vs, kt, vt) if code else H.cache(kp, vp)
    angles, _ = c.rope(d, False)
    rope = H.rope(offset(angles[0]), offset(angles[1]))
    k, v, q = c.rand(n, 2, d), c.rand(n, 2, d), c.rand(n, 4, d)
    q_out = offset(torch.zeros_like(q))
    start = torch.tensor([0, lens[0], n], dtype=torch.int32, device=DEV)
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, offset(k), offset(v), offset(q), q_out, rope, start)
    pos = torch.cat([torch.arange(L) for L in lens])
    c.ref.append(lens, lens, rotate(k, angles[0][pos], angles[1][pos], False), v)
    c.check()
    assert same(q_out, rotate(q, angles[0][pos], angles[1][pos], False))
    read = [offset(torch.zeros((2, 2, 4 * S, d), dtype=dtype)) for _ in range(2)]
    H.hils_cache_read(c.cfg, c.paged(lens), c.cache, *read)
    ql, q1 = c.rand(2, 4, 4, d), c.rand(2, 4, d)
    blank = torch.full((2, 4, 4, d), 3.0, dtype=dtype), torch.full((2, 4, 4), 3.0)
    k_sum, b_sum = offset(blank[0]), offset(blank[1])
    H.hils_build_summaries_cache(c.cfg, c.paged(lens), c.cache, offset(ql), k_sum, b_sum)
    check_summaries(c, lens, [0, 0], lambda b, ch: ql[b][:, list(ch)].double(), k_sum, b_sum, *blank)
    for b, L in enumerate(lens):
        assert same(read[0][b, :, :L], c.ref.values(0, b, L).float().to(dtype))
        assert same(read[1][b, :, :L], c.ref.values(1, b, L).float().to(dtype)) and (read[1][b, :, L:] == 0).all()
    if code:
        idx, s_sel = c.lists(lens)
        out = offset(torch.zeros((2, 4, d), dtype=dtype))
        H.hils_attn_decode_cache(c.cfg, offset(q1), c.paged(lens), c.cache, offset(idx), offset(s_sel), out)
        H.hils_sync_status()
        c.check_attention(lens, q1, idx, s_sel, out)


def test_padded_rows_are_neither_read_nor_written():
    c = Case(3, 4, 1, 128, 64, 300, BF, E4)
    angles, rope = c.rope(128, True)
    k, v, q = c.rand(40, 1, 128), c.rand(40, 1, 128), c.rand(40, 4, 128)
    k[:4], k[30:], v[30:], q[30:] = math.nan, math.nan, math.nan, math.nan
    q_out = torch.full((40, 4, 128), 9.0, dtype=BF, device=DEV)
    start = torch.tensor([4, 20, 20, 30], dtype=torch.int32, device=DEV)
    lens = [16, 0, 10]  # the second sequence is an empty slot of the batch
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV), v.to(DEV), q.to(DEV), q_out, rope, start)
    pos = torch.cat([torch.arange(16), torch.arange(10)])
    a = (angles[0][pos], angles[1][pos])
    c.ref.append(lens, [16, 0, 10], rotate(k[4:30], *a, True), v[4:30])
    c.check()
    want = torch.full((40, 4, 128), 9.0, dtype=BF)
    want[4:30] = rotate(q[4:30], *a, True)
    assert same(q_out, want)


def test_one_row_for_each_sequence_without_row_start_and_no_rows():
    c = Case(5, 2, 2, 64, 32, 100, F32, I8)
    c.fill([31, 5, 63, 90, 1])
    k, v = c.rand(5, 2, 64), c.rand(5, 2, 64)
    lens = [32, 6, 64, 91, 2]
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV), v.to(DEV))
    c.ref.append(lens, [1] * 5, k, v)
    c.check()
    none = torch.empty((0, 2, 64), device=DEV)
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, none, none, row_start=torch.zeros(6, dtype=torch.int32, device=DEV))
    c.check()


def test_one_row_each_of_more_sequences_than_a_chunk_has_tokens():
    c = Case(150, 2, 1, 64, 32, 70, F32, E4)
    rng = np.random.default_rng(4)
    old = rng.integers(0, 69, 150).tolist()
    c.fill(old)
    angles, rope = c.rope(64, False)
    k, v, q = c.rand(150, 1, 64), c.rand(150, 1, 64), c.rand(150, 2, 64)
    lens = [L + 1 for L in old]
    q_out = torch.empty_like(q, device=DEV)
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV), v.to(DEV), q.to(DEV), q_out, rope)
    a = (angles[0][torch.tensor(old)], angles[1][torch.tensor(old)])
    c.ref.append(lens, [1] * 150, rotate(k, *a, False), v)
    c.check()
    assert same(q_out, rotate(q, *a, False))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 7), (96, 12), (160, 20)])
@pytest.mark.parametrize("n", [3, 2100])
def test_any_number_of_heads(Hq, Hkv, n):
    """Fewer heads than a row has lanes, odd numbers, and more than one pass over the heads."""
    c = Case(1, Hq, Hkv, 128, 64, 2112, BF, I8)
    angles, rope = c.rope(64, True)
    c.append([n], [n], c.rand(n, Hkv, 128), c.rand(n, Hkv, 128), c.rand(n, Hq, 128), rope, angles, True)
    c.check()


def test_many_sequences():
    """More sequences than a CTA has threads."""
    B = 700
    c = Case(B, 2, 1, 64, 32, 70, F32, I8)
    rng = np.random.default_rng(2)
    news = rng.integers(0, 70, B).tolist()
    n = sum(news)
    angles, rope = c.rope(64, False)
    c.append(news, news, c.rand(n, 1, 64), c.rand(n, 1, 64), c.rand(n, 2, 64), rope, angles)
    c.check()


def expect_bad():
    with pytest.raises(H.HilsError) as e:
        H.hils_sync_status()
    assert e.value.status == H.HILS_ERR_INVALID_ARG
    H.hils_sync_status()  # cleared


@pytest.mark.parametrize("bad", ["length", "over", "few", "page", "order", "rows"])
def test_append_reports_what_it_skips(bad):
    """Sequence 1 is invalid in some way; sequence 0 is appended all the same, and nothing else changes."""
    c = Case(2, 2, 1, 64, 32, 128, F32, I8, fill=1.0)
    k, v = c.rand(80, 1, 64), c.rand(80, 1, 64)
    lens, start = [40, 40], [0, 40, 80]
    if bad == "length":
        lens[1] = 0
    elif bad == "over":
        lens[1] = 129
    elif bad == "few":
        lens[1] = 39
    elif bad == "page":
        c.table_dev[1, 0] = c.pages
    elif bad == "order":
        start = [0, 40, 20]
    else:
        start = [0, 40, 81]
    H.hils_cache_append(c.cfg, c.paged(lens), c.cache, k.to(DEV), v.to(DEV),
                        row_start=torch.tensor(start, dtype=torch.int32, device=DEV))
    expect_bad()
    c.ref.append([40, 0], [40, 0], k, v)
    if bad == "page":  # the incomplete chunk behind it goes to the tail
        for x, rows in enumerate((k, v)):
            c.ref.tail[x][1, 0, 0, :32] = rows[40:72, 0]
            c.ref.tail[x][1, 1, 0, :8] = rows[72:80, 0]
    c.check()


def test_a_position_outside_the_tables_is_reported_and_stored_unrotated():
    c = Case(1, 2, 1, 64, 32, 64, F32, None)
    angles, rope = c.rope(64, False, max_pos=8)
    k, q = c.rand(4, 1, 64), c.rand(4, 2, 64)
    q_out = torch.empty_like(q, device=DEV)
    pos = torch.tensor([0, 8, -1, 7], dtype=torch.int32)
    H.hils_cache_append(c.cfg, c.paged([4]), c.cache, k.to(DEV), k.to(DEV), q.to(DEV), q_out, rope,
                        torch.tensor([0, 4], dtype=torch.int32, device=DEV), pos.to(DEV))
    expect_bad()
    at = torch.tensor([0, 0, 0, 7])
    co, si = angles[0][at], angles[1][at]
    co[1:3], si[1:3] = 1, 0
    c.ref.append([4], [4], rotate(k, co, si, False), k)
    c.check()
    assert torch.equal(q_out.cpu(), rotate(q, co, si, False))


# -------------------------------------------------------------- reading back ---

@pytest.mark.parametrize("shape,code", FORMATS, ids=IDS)
def test_read(shape, code):
    dtype, d, S = shape
    lens = [1, S - 1, S, 5 * S + 3, 3 * S, 0]
    c = Case(6, 2, 2, d, S, 6 * S, dtype, code)
    c.fill(lens)
    rows = 4 * S + 1  # cuts the longest
    got = [torch.full((6, 2, rows, d), 3.0, dtype=dtype, device=DEV) for _ in range(2)]
    H.hils_cache_read(c.cfg, c.paged(lens), c.cache, *got)
    one = torch.full((6, 2, 6 * S + 9, d), 3.0, dtype=dtype, device=DEV)  # values only, more rows than the capacity
    H.hils_cache_read(c.cfg, c.paged(lens), c.cache, None, one)
    H.hils_sync_status()
    for b, L in enumerate(lens):
        for x in range(2):
            want = torch.full((2, rows, d), 3.0, dtype=dtype)
            want[:, :min(L, rows)] = c.ref.values(x, b, L)[:, :rows].float().to(dtype)
            assert same(got[x][b], want)
        want = torch.full((2, 6 * S + 9, d), 3.0, dtype=dtype)
        want[:, :L] = c.ref.values(1, b, L).float().to(dtype)
        assert same(one[b], want)


def test_read_reports_what_it_skips():
    c = Case(2, 1, 1, 128, 64, 256, BF, E4)
    c.fill([256, 256])
    c.table_dev[1, 2] = -1
    out = torch.full((2, 1, 256, 128), 3.0, dtype=BF, device=DEV)
    H.hils_cache_read(c.cfg, c.paged([257, 256]), c.cache, out)
    expect_bad()
    want = torch.full((2, 1, 256, 128), 3.0, dtype=BF)
    want[1] = c.ref.values(0, 1, 256).float().to(BF)
    want[1, :, 128:192] = 3.0
    assert same(out, want)


# --------------------------------------------------------------- summaries ---

def check_summaries(c, lens, first, q_lmk, k_sum, b_sum, blank_k, blank_b):
    """first: each sequence's first summarised chunk; q_lmk(b, chunks) float64 [Hq, n, d]."""
    H.hils_sync_status()
    for b, L in enumerate(lens):
        C = L // c.S
        keep = torch.ones(k_sum.shape[2], dtype=torch.bool)
        keep[first[b]:C] = False
        assert same(k_sum[b][:, keep], blank_k[b][:, keep]) and same(b_sum[b][:, keep], blank_b[b][:, keep])
        if C <= first[b]:
            continue
        k = c.ref.values(0, b, C * c.S)[:, first[b] * c.S:].reshape(c.Hkv, -1, c.S, c.d)
        ql = q_lmk(b, range(first[b], C))
        want, ent, mag, low = summaries(k, ql, c.scale)
        big = float((k.abs().amax(dim=2).repeat_interleave(c.Hq // c.Hkv, 0) * ql.abs()).sum(-1).max() * c.scale)
        wide = float((k.abs().sum(dim=3).amax(dim=2).repeat_interleave(c.Hq // c.Hkv, 0) * ql.abs().amax(dim=2)).max() * c.scale)
        rel = weights_off(c.dtype, c.code, c.d, c.S, c.S, big, wide)
        assert out_off(c.dtype, k_sum[b][:, first[b]:C], want, mag, low, rel) <= 0, b
        # H(p) = -sum p log p: each p off by `eps` of itself moves it by at most eps (H + 1), and log and exp of
        # arguments up to `big` by 2^-22 of them; the entropy's p are not rounded to digits
        eps = 2 * 2 * (c.d + 4) * 2.0 ** -24 * big + 2.0 ** -20 + (c.S + 16) * 2.0 ** -24
        if c.dtype is BF and c.code is I8:
            eps += 2 * FIXED_Q * wide
        off = (b_sum[b][:, first[b]:C].double().cpu() - ent).abs()
        assert (off <= eps * (ent + 1) + 2.0 ** -22 * big).all(), (b, off.max())


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("shape,code", CODED + [(s, None) for s in NATIVE], ids=IDS)
def test_summaries(shape, code, G):
    dtype, d, S = shape
    lens = [1, S - 1, S, 5 * S + 3, 4 * S]
    c = Case(5, 2 * G, 2, d, S, 5 * S + 7, dtype, code)
    c.fill(lens)
    C, Hq = 5, 2 * G
    q = c.rand(5, Hq, C, d)
    ks, bs = torch.full((5, Hq, C, d), 3.0, dtype=dtype), torch.full((5, Hq, C), 4.0)
    k_sum, b_sum = ks.to(DEV), bs.to(DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged(lens), c.cache, q.to(DEV), k_sum, b_sum)
    check_summaries(c, lens, [0] * 5, lambda b, ch: q[b][:, list(ch)].double(), k_sum, b_sum, ks, bs)


@pytest.mark.parametrize("code", [I8, E4, None], ids=["i8", "e4m3", "native"])
def test_summaries_of_new_chunks_with_one_query_for_a_sequence_or_for_all(code):
    c = Case(4, 8, 2, 128, 64, 640, BF, code)
    lens, start = [128, 200, 640, 63], [127, 130, 300, 62]
    c.fill(lens)
    ks, bs = torch.full((4, 8, 10, 128), 3.0, dtype=BF), torch.full((4, 8, 10), 4.0)
    first = [1, 2, 4, 0]
    old = torch.tensor(start, dtype=torch.int32, device=DEV)
    for q in (c.rand(4, 8, 128), c.rand(8, 128)):
        k_sum, b_sum = ks.to(DEV), bs.to(DEV)
        H.hils_build_summaries_cache(c.cfg, c.paged(lens), c.cache, q.to(DEV), k_sum, b_sum, old)
        check_summaries(c, lens, first, lambda b, ch: (q[b] if q.ndim == 3 else q)[:, None].double().expand(8, len(ch), 128),
                        k_sum, b_sum, ks, bs)


def test_summaries_equal_those_of_the_native_calls():
    """A native cache and hils_build_summaries_paged: the same sums in float32, another order of adding."""
    c = Case(2, 8, 2, 128, 64, 320, BF)
    c.fill([320, 130])
    q = c.rand(2, 8, 5, 128).to(DEV)
    out = [(torch.zeros((2, 8, 5, 128), dtype=BF, device=DEV), torch.zeros((2, 8, 5), device=DEV)) for _ in range(2)]
    H.hils_build_summaries_cache(c.cfg, c.paged([320, 130]), c.cache, q, *out[0])
    H.hils_build_summaries_paged(c.cfg, c.paged([320, 130]), c.dev[0][0], q, *out[1])
    H.hils_sync_status()
    k = c.ref.values(0, 0, 320).abs().max().item()
    assert (out[0][0].float() - out[1][0].float()).abs().max().item() <= 2 * k * 2.0 ** -8
    assert (out[0][1] - out[1][1]).abs().max().item() <= 2e-5


def test_summaries_of_non_finite_and_zero_blocks():
    c = Case(1, 4, 1, 128, 64, 256, BF, I8)
    k = c.rand(256, 1, 128)
    k[:64] = 0
    k[70, 0, 3] = math.inf
    c.append([256], [256], k, k)
    k_sum, b_sum = torch.zeros((1, 4, 4, 128), dtype=BF, device=DEV), torch.zeros((1, 4, 4), device=DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged([256]), c.cache, c.rand(1, 4, 4, 128).to(DEV), k_sum, b_sum)
    H.hils_sync_status()
    assert (k_sum[:, :, 0] == 0).all() and (b_sum[:, :, 0] - math.log(64)).abs().max() <= 2.0 ** -21
    assert k_sum[:, :, 1].isnan().all() and b_sum[:, :, 1].isnan().all()
    assert k_sum[:, :, 2:].isfinite().all() and b_sum[:, :, 2:].isfinite().all()


def test_summaries_report_what_they_skip():
    c = Case(3, 2, 1, 64, 32, 128, F32, E4)
    c.fill([128, 128, 128])
    c.table_dev[1, 2] = c.pages + 7
    k_sum, b_sum = torch.full((3, 2, 4, 64), 3.0, device=DEV), torch.full((3, 2, 4), 3.0, device=DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged([0, 128, 129]), c.cache, c.rand(3, 2, 4, 64).to(DEV), k_sum, b_sum)
    expect_bad()
    done = (k_sum != 3.0).any(dim=-1).any(dim=1)
    assert done.tolist() == [[False] * 4, [True, True, False, True], [False] * 4]


# --------------------------------------------------------------- attention ---

@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("shape,code", CODED, ids=CODED_IDS)
def test_attention(shape, code, G):
    """Lengths of one token to many chunks; lists that are full, part full and empty."""
    dtype, d, S = shape
    lens = [1, S - 1, S, S + 1, 2 * S, 3 * S, 5 * S + 7, 20 * S, 19 * S + 1]
    B = len(lens)
    c = Case(B, 2 * G, 2, d, S, 20 * S, dtype, code, W=2 * S, K=7)
    c.fill(lens)
    q = c.rand(B, 2 * G, d, std=1.5)
    idx, s_sel = c.lists(lens)
    out = torch.full((B, 2 * G, d), math.nan, dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    c.check_attention(lens, q, idx, s_sel, out)


@pytest.mark.parametrize("K,W", [(1, 64), (64, 64), (64, 2048), (16, 512), (3, 1024)])
@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
def test_attention_list_lengths_and_windows(code, K, W):
    lens = [100 * 64, 97 * 64 + 33, W, W + 65]
    c = Case(4, 4, 1, 128, 64, 100 * 64, BF, code, W=W, K=K)
    c.fill(lens)
    q = c.rand(4, 4, 128)
    idx, s_sel = c.lists(lens)
    out = torch.empty((4, 4, 128), dtype=BF, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    c.check_attention(lens, q, idx, s_sel, out)


@pytest.mark.parametrize("B", [2, 20, 45, 90, 300, 520, 1000, 1900])
@pytest.mark.parametrize("dtype,d,S,code,G", [(BF, 128, 64, I8, 2), (BF, 128, 64, E4, 4), (F32, 64, 32, I8, 1)],
                         ids=["bf16-i8", "bf16-e4m3", "f32-i8"])
def test_attention_and_summaries_of_any_number_of_sequences(B, dtype, d, S, code, G):
    """One launch shape after the other: clusters of CTAs, one CTA of 12 to 3 warps, several waves of four; summaries
    over more sequences than one block of CTAs takes."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 5 * S, B).tolist()
    c = Case(B, G, 1, d, S, 5 * S, dtype, code, W=2 * S, K=3)
    c.fill(lens)
    q, ql = c.rand(B, G, d), c.rand(B, G, 5, d)
    idx, s_sel = c.lists(lens)
    out = torch.full((B, G, d), math.nan, dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    ks, bs = torch.full((B, G, 5, d), 3.0, dtype=dtype), torch.full((B, G, 5), 4.0)
    k_sum, b_sum = ks.to(DEV), bs.to(DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged(lens), c.cache, ql.to(DEV), k_sum, b_sum)
    H.hils_sync_status()
    some = sorted({0, 1, B // 3, B // 2, B - 2, B - 1} | set(rng.integers(0, B, 12).tolist()))
    for b in some:
        k, v = c.ref.values(0, b, lens[b]), c.ref.values(1, b, lens[b])
        want, mag, low, big, wide = attend(q[b].double(), k, v, idx[b].tolist(), s_sel[b].double(), S, c.W, c.scale)
        rel = weights_off(dtype, code, d, S, 3 * S + c.W, big, wide)
        assert out_off(dtype, out[b], want, mag, low, rel) <= 0, (b, lens[b])
    assert out.isfinite().all()
    check_summaries(c, lens, [0] * B, lambda b, ch: ql[b][:, list(ch)].double(), k_sum, b_sum, ks, bs)


@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
def test_attention_with_more_units_than_a_warp_looks_ahead(code):
    """512 sequences of 64 chosen chunks and a window of 32: three warps each, 32 units a warp."""
    B, L = 512, 100 * 64 - 5
    c = Case(1, 2, 1, 128, 64, 100 * 64, BF, code, W=32 * 64, K=64)
    c.fill([L])
    idx, s_sel = c.lists([L])
    q = c.rand(B, 2, 128)
    cfg = H.make_config(B, 100 * 64, 2, 1, 128, 64, 32 * 64, 64, BF)
    # every sequence reads the same pages and the same tail rows
    tails = [t.expand(B, *t.shape[1:]).contiguous() for t in c.dev[2]]
    cache = H.cache(*c.dev[0], *c.dev[1], *tails)
    table = c.table_dev.expand(B, -1).contiguous()
    pg = H.paged(torch.full((B,), L, dtype=torch.int32, device=DEV), table, c.pages)
    out = torch.empty((B, 2, 128), dtype=BF, device=DEV)
    H.hils_attn_decode_cache(cfg, q.to(DEV), pg, cache, idx.expand(B, -1, -1).contiguous().to(DEV),
                             s_sel.expand(B, -1, -1).contiguous().to(DEV), out)
    H.hils_sync_status()
    k, v = c.ref.values(0, 0, L), c.ref.values(1, 0, L)
    for b in (0, 1, 255, 511):
        want, mag, low, big, wide = attend(q[b].double(), k, v, idx[0].tolist(), s_sel[0].double(), 64, c.W, c.scale)
        rel = weights_off(BF, code, 128, 64, 96 * 64, big, wide)
        assert out_off(BF, out[b], want, mag, low, rel) <= 0, b


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attention_with_large_and_small_values(dtype):
    """Sharp softmaxes, queries and blocks of very different sizes, and score weights far apart."""
    c = Case(3, 8, 2, 128, 64, 640, dtype, I8, W=128, K=4)
    lens = [640, 333, 500]
    n = sum(lens)
    size = 10.0 ** torch.empty(n, 1, 1).uniform_(-3, 0.5, generator=c.gen)
    c.append(lens, lens, (c.rand(n, 2, 128) * size).to(dtype), (c.rand(n, 2, 128) * 10.0 ** torch.empty(n, 2, 1).uniform_(-20, 20, generator=c.gen)).to(dtype))
    q = (c.rand(3, 8, 128) * torch.logspace(-4, 1, 8)[None, :, None]).to(dtype)
    idx, s_sel = c.lists(lens)
    s_sel[1] *= 30
    s_sel[2, :, 0] = -math.inf
    out = torch.empty((3, 8, 128), dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    c.check_attention(lens, q, idx, s_sel, out)


@pytest.mark.parametrize("dtype,code,G", [(BF, I8, 4), (BF, I8, 8), (BF, E4, 4), (F32, I8, 2)])
def test_attention_over_blocks_of_zeros_and_queries_of_zeros(dtype, code, G):
    """Scales of zero (all logits of the block alike, nothing added to the sums), a query of zeros and a tiny one, and
    a whole context of zeros."""
    c = Case(2, G, 1, 128, 64, 640, dtype, code, W=128, K=4)
    lens = [600, 640]
    k, v = c.rand(1240, 1, 128), c.rand(1240, 1, 128)
    k[64:128] = 0
    v[128:192] = 0
    k[512:540], v[530:560] = 0, 0
    k[600:], v[600:] = 0, 0
    c.append(lens, lens, k, v)
    idx, s_sel = c.lists(lens)
    idx[0, 0] = torch.tensor([0, 1, 2, 5])
    q = c.rand(2, G, 128)
    q[0, 0], q[0, 1] = 0, q[0, 1] * 2.0 ** -120
    out = torch.full((2, G, 128), math.nan, dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    c.check_attention(lens, q, idx, s_sel, out)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_the_smallest_blocks_that_are_held(dtype, code):
    """Values of 2^-109 to 2^-100: a scale over a sum of weights is below the normal range, the sums are not."""
    c = Case(1, 8, 2, 128, 64, 640, dtype, code, W=128, K=3)
    k, v = c.rand(600, 2, 128), c.rand(600, 2, 128)
    k[:300] *= 2.0 ** -109
    v *= 2.0 ** -109
    v[300:] *= 2.0 ** 9
    c.append([600], [600], k, v)
    idx, s_sel = c.lists([600])
    q, ql = c.rand(1, 8, 128), c.rand(1, 8, 10, 128)
    out = torch.empty((1, 8, 128), dtype=dtype, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged([600]), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    blank = torch.full((1, 8, 10, 128), 3.0, dtype=dtype), torch.full((1, 8, 10), 3.0)
    k_sum, b_sum = blank[0].to(DEV), blank[1].to(DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged([600]), c.cache, ql.to(DEV), k_sum, b_sum)
    H.hils_sync_status()
    assert (out != 0).all() and (k_sum[:, :, :4] != 0).float().mean() > 0.9
    c.check_attention([600], q, idx, s_sel, out)
    check_summaries(c, [600], [0], lambda b, ch: ql[b][:, list(ch)].double(), k_sum, b_sum, *blank)


def test_codes_and_scales_that_no_append_makes():
    """A pool filled elsewhere: codes of -128, scales that are negative, very small and very large."""
    c = Case(1, 8, 2, 128, 64, 640, BF, I8, W=128, K=6)
    c.fill([640])
    for x in range(2):
        c.ref.pool[x][:, :, ::3, ::5] = -128
        c.ref.scale[x][int(c.table[0, 1])] = -0.02
        c.ref.scale[x][int(c.table[0, 2])] = 2.0 ** -130
    c.ref.scale[1][int(c.table[0, 3])] = 2.0 ** 100
    for got, want in zip(c.dev, (c.ref.pool, c.ref.scale)):
        for x in range(2):
            got[x].copy_(want[x])
    idx = torch.arange(6, dtype=torch.int32).expand(1, 2, 6).contiguous()
    s_sel = 3 + c.rand(1, 8, 6).float()
    q = c.rand(1, 8, 128)
    out = torch.empty((1, 8, 128), dtype=BF, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged([640]), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    ql = c.rand(1, 8, 10, 128)
    blank = torch.full((1, 8, 10, 128), 3.0, dtype=BF), torch.full((1, 8, 10), 3.0)
    k_sum, b_sum = blank[0].to(DEV), blank[1].to(DEV)
    H.hils_build_summaries_cache(c.cfg, c.paged([640]), c.cache, ql.to(DEV), k_sum, b_sum)
    H.hils_sync_status()
    c.check_attention([640], q, idx, s_sel, out)
    check_summaries(c, [640], [0], lambda b, ch: ql[b][:, list(ch)].double(), k_sum, b_sum, *blank)


def test_attention_reads_no_masked_place():
    """NaN in every place that the token does not attend: unchosen chunks, tail rows behind its length, the other
    tail slot, unused pages."""
    c = Case(2, 4, 1, 128, 64, 640, BF, E4, W=128, K=3)
    lens = [640 - 20, 600]
    c.fill(lens)
    idx, s_sel = c.lists(lens)
    read = set()
    for b, L in enumerate(lens):
        cur = (L - 1) // 64
        keep = set(idx[b, 0].tolist()) | {cur, cur - 1}
        read |= {int(c.table[b, x]) for x in keep if 0 <= x < L // 64}
        for t in c.dev[2]:
            t[b, (cur + 1) & 1] = math.nan
            t[b, cur & 1, :, L % 64:] = math.nan
    for p in range(c.pages):
        if p not in read:
            for x in range(2):
                c.dev[1][x][p] = math.nan
                c.dev[0][x].view(torch.uint8)[p] = 0x7f
    q = c.rand(2, 4, 128)
    out = torch.empty((2, 4, 128), dtype=BF, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    c.check_attention(lens, q, idx, s_sel, out)


@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("place", ["chosen", "window", "tail", "only"])
def test_attention_over_a_non_finite_block_is_nan(place, where):
    c = Case(2, 4, 1, 128, 64, 640, BF, I8, W=128, K=3)
    lens = [620, 620] if place != "only" else [64, 64]  # only: the whole window is that block
    n = lens[0]
    k, v = c.rand(2 * n, 1, 128), c.rand(2 * n, 1, 128)
    at = {"chosen": 70, "window": 8 * 64 + 3, "tail": 610, "only": 5}[place]
    (k if where == "key" else v)[at, 0, 17] = math.nan  # of the first sequence
    c.append(lens, lens, k, v)
    idx, s_sel = c.lists(lens)
    if place != "only":
        idx[:, 0] = torch.tensor([0, 1, 4])
    q = c.rand(2, 4, 128)
    out = torch.zeros((2, 4, 128), dtype=BF, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    H.hils_sync_status()
    bad = out[0].isnan()
    assert (bad.all() if where == "key" or place != "tail" else bad[:, 17].all()) and out[1].isfinite().all()


def test_attention_reports_what_it_skips():
    """A list entry that is no candidate, one that does not ascend, a page outside the pool, and lengths outside the
    capacity, whose rows are left as they were."""
    c = Case(4, 4, 1, 128, 64, 640, BF, I8, W=128, K=4)
    lens = [640, 500, 640, 640]
    c.fill(lens)
    q = c.rand(4, 4, 128)
    idx, s_sel = c.lists(lens)
    idx[0, 0] = torch.tensor([1, 8, 3, -1])  # 8 is in the window; 3 is below it
    s_sel[0] = 2.0
    accepted = idx.clone()
    accepted[0, 0] = torch.tensor([1, -1, 3, -1])
    bad = idx.clone()
    out = torch.full((4, 4, 128), 5.0, dtype=BF, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged([640, 500, 0, 641]), c.cache, bad.to(DEV), s_sel.to(DEV), out)
    expect_bad()
    assert (out[2:] == 5.0).all()
    # the list rule: an entry counts against later ones even if it is dropped
    accepted[0, 0] = torch.tensor([1, -1, -1, -1])
    c.check_attention(lens[:2], q, idx, s_sel, out, accepted)
    c.table_dev[1, 7] = c.pages  # in the window of sequence 1
    H.hils_attn_decode_cache(c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), out)
    expect_bad()


@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
def test_pools_past_32_bit_offsets(code):
    """Pages whose element offsets pass 2^31 and, for the tail of a page table's end, 2^32."""
    pages, Hkv, S, d = 66000, 8, 64, 128  # 65536 elements a page
    cfg = H.make_config(1, 512, 16, Hkv, d, S, 128, 2, BF)
    small = Case(1, 16, Hkv, d, S, 512, BF, code, W=128, K=2)
    pools = [torch.zeros((pages, Hkv, S, d), dtype=torch.uint8, device=DEV).view(code) for _ in range(2)]
    scales = [torch.zeros((pages, Hkv), device=DEV) for _ in range(2)]
    tails = [torch.zeros((1, 2, Hkv, S, d), dtype=BF, device=DEV) for _ in range(2)]
    cache = H.cache(*pools, *scales, *tails)
    table = torch.tensor([[65999, 0, 40000, 33000, 65537, 32767, 32768, 65990]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([500], dtype=torch.int32, device=DEV)
    pg = H.paged(lens, table, pages)
    k, v = small.rand(500, Hkv, d), small.rand(500, Hkv, d)
    H.hils_cache_append(cfg, pg, cache, k.to(DEV), v.to(DEV), row_start=torch.tensor([0, 500], dtype=torch.int32, device=DEV))
    small.append([500], [500], k, v)
    got = [torch.zeros((1, Hkv, 500, d), dtype=BF, device=DEV) for _ in range(2)]
    H.hils_cache_read(cfg, pg, cache, *got)
    small.check()
    for x in range(2):
        assert same(got[x][0], small.ref.values(x, 0, 500).float().to(BF))
    q, ql = small.rand(1, 16, d), small.rand(1, 16, 8, d)
    idx, s_sel = small.lists([500])
    outs, sums = [], []
    for p, ca in ((pg, cache), (small.paged([500]), small.cache)):
        out = torch.zeros((1, 16, d), dtype=BF, device=DEV)
        ks, bs = torch.zeros((1, 16, 8, d), dtype=BF, device=DEV), torch.zeros((1, 16, 8), device=DEV)
        H.hils_attn_decode_cache(cfg, q.to(DEV), p, ca, idx.to(DEV), s_sel.to(DEV), out)
        H.hils_build_summaries_cache(cfg, p, ca, ql.to(DEV), ks, bs)
        outs.append(out)
        sums.append((ks, bs))
    H.hils_sync_status()
    assert same(outs[0], outs[1]) and same(sums[0][0], sums[1][0]) and same(sums[0][1], sums[1][1])
    small.check_attention([500], q, idx, s_sel, outs[0])


# ------------------------------------------------- the run of them together ---

@pytest.mark.parametrize("fmt", ["native", "int8", "e4m3"])
def test_prompt_and_decode_steps(fmt):
    """A ragged batch through CacheDecode: prompts, then decode steps across chunk borders.  Each step's scores,
    selection and output are checked on the values that the cache holds, by the oracle."""
    import oracle
    from tests.parity import check_selection, forced_s_sel

    B, Hq, Hkv, d, S, W, K, cap = 3, 8, 2, 128, 64, 128, 4, 2048
    cfg = H.make_config(B, cap, Hq, Hkv, d, S, W, K, BF)
    code = {"native": None, "int8": I8, "e4m3": E4}[fmt]
    model = Case(B, Hq, Hkv, d, S, cap, BF, code, W=W, K=K)
    (cos, sin), rope = model.rope(d, False)
    lens = [1000, 62, 1919]
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    dec = H.CacheDecode(cfg, seq_lens, model.table_dev, model.pages, fmt, rope)
    q_lmk = model.rand(B, Hq, cap // S, d)
    n = sum(lens)
    k, v = model.rand(n, Hkv, d), model.rand(n, Hkv, d)
    pos = torch.cat([torch.arange(L) for L in lens])
    dec.append(k.to(DEV), v.to(DEV), q_lmk.to(DEV),
               row_start=torch.tensor([0, 1000, 1062, n], dtype=torch.int32, device=DEV))
    model.ref.append(lens, lens, rotate(k, cos[pos], sin[pos], False), v)
    for step in range(5):
        old = seq_lens.clone()
        seq_lens += 1
        lens = [L + 1 for L in lens]
        k, v, q = model.rand(B, Hkv, d), model.rand(B, Hkv, d), model.rand(B, Hq, d)
        pos = torch.tensor(lens) - 1
        q_out = torch.empty_like(q, device=DEV)
        ql = torch.stack([q_lmk[b, :, max(0, L // S - 1)] for b, L in enumerate(lens)])
        dec.append(k.to(DEV), v.to(DEV), ql.to(DEV), q.to(DEV), q_out, from_lens=old)
        model.ref.append(lens, [1] * B, rotate(k, cos[pos], sin[pos], False), v)
        out = dec.step(q_out)
        H.hils_sync_status()
        for b, L in enumerate(lens):
            kk, vv = (model.ref.values(x, b, L)[None].numpy() for x in range(2))
            dm = oracle.Dims(B=1, Hq=Hq, Hkv=Hkv, N=L, d=d, S=S, W=W, K=K, nq=1, q_pos0=L - 1)
            qb = q_out[b:b + 1, :, None].float().cpu().numpy()
            ks, bs = oracle.summaries(dm, kk, q_lmk[b:b + 1, :, :L // S].float().numpy())
            if L >= S:
                assert np.abs(dec.b_sum[b:b + 1, :, :L // S].cpu().numpy() - bs).max() <= 2e-5
            _, _, s_all, g_all = oracle.select(dm, [(0, L - 1)], qb, k_sum=ks, b_sum=bs, want_all=True)
            idx = dec.idx[b:b + 1].cpu().numpy().astype(np.int64)
            check_selection(idx, g_all, K)
            ref = oracle.attend(dm, [(0, L - 1)], qb, kk, vv, idx, forced_s_sel(idx, s_all, Hq // Hkv))
            assert np.abs(out[b:b + 1].float().cpu().numpy() - ref).max() <= 1.5e-2


def test_prefill_over_what_the_cache_holds():
    """A prompt appended and read back feeds the prefill: rows are those that decode will read."""
    N, Hq, Hkv, d, S, W, K = 1024, 4, 1, 128, 64, 128, 4
    c = Case(1, Hq, Hkv, d, S, N, BF, I8, W=W, K=K)
    angles, rope = c.rope(d, False)
    q = torch.empty((1, Hq, N, d), dtype=BF, device=DEV)
    kv = [torch.empty((1, Hkv, N, d), dtype=BF, device=DEV) for _ in range(2)]
    rows = c.rand(N, Hq + 2 * Hkv, d).to(DEV)
    H.hils_cache_append(c.cfg, c.paged([N]), c.cache, rows[:, Hq:Hq + 1], rows[:, Hq + 1:], rows[:, :Hq],
                        q[0].transpose(0, 1), rope, torch.tensor([0, N], dtype=torch.int32, device=DEV))
    H.hils_cache_read(c.cfg, c.paged([N]), c.cache, *kv)
    q_lmk = c.rand(1, Hq, N // S, d).to(DEV)
    pre = H.Prefill(c.cfg, DEV)
    out = pre.run(q, *kv, q_lmk)
    # the last token as a decode step with the prefill's list and scores
    last = torch.empty((1, Hq, d), dtype=BF, device=DEV)
    H.hils_attn_decode_cache(c.cfg, q[:, :, -1].contiguous(), c.paged([N]), c.cache, pre.idx[:, :, -1].contiguous(),
                             pre.s_sel[:, :, -1].contiguous(), last)
    H.hils_sync_status()
    # both are within the bf16 bound of the same sums; the prefill's rows round to bf16 once more (2^-8 of logit
    # and value: |logit| <= 4 or so here), so the shared tolerance of bf16 outputs applies
    assert (last.float() - out[:, :, -1].float()).abs().max().item() <= 1.5e-2


def _step_case(fmt_code):
    c = Case(2, 8, 2, 128, 64, 640, BF, fmt_code, W=128, K=3)
    lens = [511, 300]
    c.fill(lens)
    angles, rope = c.rope(128, False)
    return c, lens, rope


@pytest.mark.parametrize("code", [I8, E4], ids=["i8", "e4m3"])
def test_a_step_captured_into_a_graph_and_replayed(code):
    """The captured calls read lengths, rows and lists from device memory at each replay."""
    eager, lens, rope = _step_case(code)
    graph_c, _, _ = _step_case(code)
    B, Hq, Hkv, d = 2, 8, 2, 128

    def buffers():
        return dict(k=torch.empty((B, Hkv, d), dtype=BF, device=DEV), v=torch.empty((B, Hkv, d), dtype=BF, device=DEV),
                    q=torch.empty((B, Hq, d), dtype=BF, device=DEV), qo=torch.empty((B, Hq, d), dtype=BF, device=DEV),
                    ql=torch.empty((B, Hq, d), dtype=BF, device=DEV), out=torch.empty((B, Hq, d), dtype=BF, device=DEV),
                    ks=torch.zeros((B, Hq, 10, d), dtype=BF, device=DEV), bs=torch.zeros((B, Hq, 10), device=DEV),
                    lens=torch.zeros(B, dtype=torch.int32, device=DEV), old=torch.zeros(B, dtype=torch.int32, device=DEV),
                    idx=torch.full((B, Hkv, 3), -1, dtype=torch.int32, device=DEV),
                    s=torch.zeros((B, Hq, 3), device=DEV))

    def step(c, x):
        pg = H.paged(x["lens"], c.table_dev, c.pages)
        H.hils_cache_append(c.cfg, pg, c.cache, x["k"], x["v"], x["q"], x["qo"], rope)
        H.hils_build_summaries_cache(c.cfg, pg, c.cache, x["ql"], x["ks"], x["bs"], x["old"])
        H.hils_attn_decode_cache(c.cfg, x["qo"], pg, c.cache, x["idx"], x["s"], x["out"])

    a, z = buffers(), buffers()
    z["lens"].copy_(torch.tensor(lens))
    z["old"].copy_(torch.tensor(lens))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for x in z.values():  # a warm-up on this step's own inputs would append; run the attention only
            pass
        z["idx"].fill_(-1)
        H.hils_attn_decode_cache(graph_c.cfg, z["q"].zero_(), H.paged(z["lens"], graph_c.table_dev, graph_c.pages),
                                 graph_c.cache, z["idx"], z["s"], z["out"])
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(graph_c, z)
    for i in range(4):
        old = torch.tensor(lens, dtype=torch.int32)
        lens = [L + 1 for L in lens]
        idx, s_sel = eager.lists(lens, seed=i)
        new = dict(k=eager.rand(B, Hkv, d), v=eager.rand(B, Hkv, d), q=eager.rand(B, Hq, d), ql=eager.rand(B, Hq, d),
                   lens=torch.tensor(lens, dtype=torch.int32), old=old, idx=idx, s=s_sel)
        for x in (a, z):
            for n, t in new.items():
                x[n].copy_(t)
        step(eager, a)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        H.hils_sync_status()
        for n in ("qo", "out", "ks", "bs"):
            assert same(a[n], z[n]), (i, n)
        for x, y in zip(eager.dev, graph_c.dev):
            assert same(x[0], y[0]) and same(x[1], y[1])


def test_two_streams_at_once_and_repeats_bit_for_bit():
    c = Case(8, 32, 4, 128, 64, 4096, BF, I8, W=512, K=16)
    lens = [4096, 4000, 3333, 2048, 4095, 1, 700, 4096]
    c.fill(lens)
    q = c.rand(8, 32, 128).to(DEV)
    idx, s_sel = (t.to(DEV) for t in c.lists(lens))
    q2 = (q.flip(0)).contiguous()
    pg = c.paged(lens)
    want = []
    for x in (q, q2):
        out = torch.empty_like(x)
        H.hils_attn_decode_cache(c.cfg, x, pg, c.cache, idx, s_sel, out)
        want.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(q) for _ in range(2)]
    for _ in range(20):
        for st, x, out in zip(streams, (q, q2), outs):
            H.hils_attn_decode_cache(c.cfg, x, pg, c.cache, idx, s_sel, out, stream=st)
    torch.cuda.synchronize()
    H.hils_sync_status()
    assert same(outs[0], want[0]) and same(outs[1], want[1])


def test_a_wait_that_runs_out_is_reported():
    """The test hook keeps the tile copies from being issued: the bounded waits run out, and the calls work again after."""
    c = Case(2, 8, 2, 128, 64, 640, BF, I8, W=128, K=3)
    lens = [640, 300]
    c.fill(lens)
    idx, s_sel = c.lists(lens)
    q, q_lmk = c.rand(2, 8, 128), c.rand(2, 8, 10, 128).to(DEV)
    args = (c.cfg, q.to(DEV), c.paged(lens), c.cache, idx.to(DEV), s_sel.to(DEV), torch.empty((2, 8, 128), dtype=BF, device=DEV))
    sums = [torch.zeros((2, 8, 10, 128), dtype=BF, device=DEV), torch.zeros((2, 8, 10), device=DEV)]
    H.hils_sync_status()
    for run in (lambda: H.hils_attn_decode_cache(*args),
                lambda: H.hils_build_summaries_cache(c.cfg, c.paged(lens), c.cache, q_lmk, *sums)):
        try:
            H.hils_set_wait_budget(2_000_000)  # about a millisecond
            H.hils_set_fault_injection(1)
            run()
        finally:
            H.hils_set_fault_injection(0)
            H.hils_set_wait_budget(0)
        with pytest.raises(H.HilsError) as e:
            H.hils_sync_status()
        assert e.value.status == H.HILS_ERR_TIMEOUT
        run()
        H.hils_sync_status()
    c.check_attention(lens, q, idx, s_sel, args[-1])
