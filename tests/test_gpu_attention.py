"""Attention over the paged quantized cache against the formula in 64 bits.

Bars, from the arithmetic (u = 2^-8, half a step of bf16 relative to the value):
  * the output is rounded once: u |out|;
  * each softmax weight is rounded to bf16 for the product: u sum_j p_j |v_j|;
  * a score is off by at most e = scale * max_j (sum_d |q'_d k_jd|) * (2^-22 D^(1/2) + u [q' rounded,
    with factors only]) -- fp32 sums of D products err by less than 2^-24 D^(1/2) in a
    typical and 2^-24 D in the worst order; 2^-22 D^(1/2) covers both up to D = 256 -- and
    errors of the exponential's 2^-22; weights then change by a factor within exp(+-2 e);
  * the fp32 sums over tokens: 2^-16 sum_j p_j |v_j| covers 2^-24 times a few hundred partial sums.
  * products p v are held in units of 2^-32 (the header's range statement), so one below 2^-94
    (fp32's smallest normal 2^-126 times 2^32) may be lost: at most L 2^-94 for L tokens.
With output factors the bounds of a row go through |P_o|.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def bat():
    import w4a4_bit_gemm_b200 as m
    m.lib()
    return m


def _factors(g, nb, s=8):
    t = 32 // s
    A = torch.eye(s) + 0.1 * torch.randn(s, s, generator=g)
    B = torch.eye(t) + 0.1 * torch.randn(nb, t, t, generator=g)
    return A.cuda().contiguous(), B.cuda().contiguous()


def _dense(A, B):
    return [torch.kron(b.double(), A.double()) for b in B]


def _apply(x, P):
    return torch.cat([x[..., 32 * i:32 * i + 32] @ m for i, m in enumerate(P)], -1)


class Setup:
    """Caches filled through bat_kv_quantize (rows no sequence owns hold NaN), and the call."""

    # capacity: tokens the page table has room for; with room for many, chunks go to the tile kernel
    def __init__(self, bat, seqs, Hq, H, D, fmt, page, seed=0, q_pad=0, qf=None, of=None, extra_rows=0, kv_scale=1.0,
                 capacity=1 << 20):
        g = torch.Generator().manual_seed(seed)
        self.bat, self.seqs, self.Hq, self.H, self.D, self.page = bat, seqs, Hq, H, D, page
        pages = [max(1, -(-L // page)) for _, L in seqs]
        self.max_pages = max(max(pages), capacity // page)
        pool = sum(pages) + 2
        perm = torch.randperm(pool, generator=g).tolist()
        table = torch.full((len(seqs), self.max_pages), 2 ** 30, dtype=torch.int32)  # unused entries: garbage
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.table = table.cuda()
        self.slots = pool * page
        eyeA, eyeB = torch.eye(8).cuda(), torch.eye(4).repeat(D // 32, 1, 1).cuda()
        self.caches, self.vals = [], []
        for _ in range(2):
            c = bat.KVCache.empty(self.slots, H, D, fmt)
            c.codes.fill_(0x7F)
            c.scales.fill_(255)
            vals = []
            for b, (_, L) in enumerate(seqs):
                if L == 0:
                    vals.append(None)
                    continue
                j = torch.arange(L)
                slot = (table[b, j // page].long() * page + j % page).cuda()
                x = (torch.randn(L, H, D, generator=g) * kv_scale).bfloat16().cuda()
                bat.bat_kv_quantize(x, eyeA, eyeB, slot, c)
                vals.append(bat.bat_kv_dequantize(c, slot).double())
            self.caches.append(c)
            self.vals.append(vals)
        self.T = sum(n for n, _ in seqs)
        rows = self.T + extra_rows
        wide = (1.5 * torch.randn(rows, Hq * D + q_pad, generator=g)).bfloat16().cuda()
        self.q = wide[:, :Hq * D].unflatten(1, (Hq, D))
        self.kv_lens = torch.tensor([L for _, L in seqs], dtype=torch.int32).cuda()
        self.q_starts = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32).cuda()
        self.qf = _factors(g, D // 32, qf) if qf else None
        self.of = _factors(g, D // 32, of) if of else None

    def call(self, **kw):
        a = dict(q_factors=self.qf, out_factors=self.of)
        a.update(kw)
        mq = a.pop("max_q_len", max(n for n, _ in self.seqs) or 1)
        return self.bat.bat_kv_attention(self.q, *self.caches, self.table, self.kv_lens, self.q_starts, self.page,
                                         mq, **a)

    def check(self, out, lse=None, window=0, sinks=0, scale=None):
        D, G = self.D, self.Hq // self.H
        scale = D ** -0.5 if scale is None else scale
        q = self.q.double()
        if self.qf:
            q = _apply(q, _dense(*self.qf))
        at = 0
        for b, (n, L) in enumerate(self.seqs):
            if n == 0:
                continue
            got = out[at:at + n].double()
            if L == 0:
                assert torch.all(got == 0)
                if lse is not None:
                    assert torch.all(torch.isneginf(lse[at:at + n]))
                at += n
                continue
            pos = torch.arange(L - n, L).cuda()[:, None]
            j = torch.arange(L).cuda()[None]
            see = j <= pos
            if window:
                see = see & ((j > pos - window) | (j < sinks))
            for h in range(self.H):
                k, v = self.vals[0][b][:, h], self.vals[1][b][:, h]
                qq = q[at:at + n, h * G:(h + 1) * G]
                x = torch.einsum("tgd,kd->tgk", qq, k) * scale
                x = x.masked_fill(~see[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                p = torch.where(torch.isneginf(x), 0.0, torch.exp(x - z[..., None]).nan_to_num(0.0))
                ref, mag = p @ v, p @ v.abs()
                big = (torch.einsum("tgd,kd->tgk", qq.abs(), k.abs()) * abs(scale)).masked_fill(~see[:, None], 0).amax(-1)
                e = big * (2 ** -22 * math.sqrt(D) + (U if self.qf else 0.0)) + 2 ** -22
                bound = mag * (U + 2 ** -16 + torch.expm1(2 * e)[..., None])
                bound = bound + L * 2.0 ** -94
                if self.of:
                    P = _dense(*self.of)
                    ref, bound = _apply(ref, P), _apply(bound, [m.abs() for m in P])
                bound = bound * (1 + U) + U * ref.abs()
                err = (got[:, h * G:(h + 1) * G] - ref).abs()
                bad = ~(err <= bound)
                assert not bad.any(), (b, h, torch.argwhere(bad)[:4].tolist(), (err / bound).max().item())
                if lse is not None:
                    gl = lse[at:at + n, h * G:(h + 1) * G].double()
                    empty = torch.isneginf(z)
                    assert torch.equal(torch.isneginf(gl), empty)
                    d = (gl - z).abs()[~empty]
                    assert torch.all(d <= e[~empty] + 2 ** -20 + 2 ** -22 * z[~empty].abs()), d.max()
            at += n


CASES = [
    # seqs [(new, cached)], Hq, H, D, fmt, page, keyword arguments
    ([(1, 1)], 1, 1, 32, "mxfp8", 1, {}),
    ([(1, 1000)], 32, 8, 128, "mxfp8", 16, {}),
    ([(1, 257), (1, 1), (1, 128), (1, 129), (1, 3000)], 8, 2, 64, "mxfp8", 24, {}),
    ([(1, 700), (0, 50), (1, 0), (3, 2), (1, 2500)], 6, 2, 96, "mxfp4", 7, {}),
    ([(5, 333), (2, 2), (1, 1), (4, 4000)], 28, 4, 128, "mxfp4", 64, {}),
    ([(1, 515), (2, 999)], 24, 2, 128, "mxfp8", 32, {}),            # 12 heads to a KV head
    ([(1, 515), (2, 99)], 40, 1, 64, "mxfp4", 32, {}),              # 40 heads to a KV head
    ([(1, 1025), (3, 77)], 8, 1, 256, "mxfp8", 16, {}),
    ([(1, 1025), (3, 77)], 10, 1, 160, "mxfp4", 16, {}),
    ([(1, 5000), (2, 40), (1, 300)], 8, 2, 128, "mxfp8", 16, {"window": 100}),
    ([(1, 5000), (2, 40), (1, 300)], 8, 2, 128, "mxfp8", 16, {"window": 100, "sinks": 4}),
    ([(1, 5000), (7, 260)], 8, 2, 64, "mxfp4", 16, {"window": 1, "sinks": 130}),
    ([(1, 900), (3, 70)], 8, 2, 128, "mxfp8", 16, {"window": 1}),
    ([(64, 64)], 4, 2, 64, "mxfp8", 16, {}),
    ([(200, 200), (33, 700), (1, 50), (130, 131)], 8, 2, 128, "mxfp8", 16, {}),
    ([(300, 1000), (17, 400)], 12, 4, 64, "mxfp4", 24, {}),
    ([(150, 400)], 7, 1, 96, "mxfp8", 5, {}),
    ([(150, 400), (20, 10)], 4, 1, 256, "mxfp4", 64, {}),
    ([(150, 400), (20, 10)], 4, 4, 192, "mxfp8", 64, {}),
    ([(600, 900), (5, 1200)], 8, 2, 128, "mxfp8", 64, {"window": 64, "sinks": 3}),
    ([(600, 900), (500, 500)], 4, 2, 64, "mxfp4", 64, {"window": 257, "sinks": 0}),
    ([(257, 2000)], 4, 1, 128, "mxfp4", 128, {"window": 300, "sinks": 200}),
    ([(130, 130), (2, 5)], 64, 1, 32, "mxfp8", 16, {}),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_matches_formula(bat, case):
    seqs, Hq, H, D, fmt, page, kw = CASES[case]
    s = Setup(bat, seqs, Hq, H, D, fmt, page, seed=case)
    lse = torch.empty(s.T, Hq, dtype=torch.float32, device="cuda")
    out = s.call(lse=lse, **kw)
    torch.cuda.synchronize()
    s.check(out, lse, **kw)
    assert bat.bat_device_error() == 0


@pytest.mark.parametrize("case", [3, 8, 14, 15, 16, 17, 18, 19, 20, 21, 22])
def test_attention_chunks_on_the_row_kernel(bat, case):
    """The same chunks where the call may expect single tokens, and with a table of the lengths' size."""
    seqs, Hq, H, D, fmt, page, kw = CASES[case]
    s = Setup(bat, seqs, Hq, H, D, fmt, page, seed=200 + case, qf=8, of=8, capacity=0)
    lse = torch.empty(s.T, Hq, dtype=torch.float32, device="cuda")
    s.check(s.call(max_q_len=1, lse=lse, **kw), None, **kw)
    s.check(s.call(**kw), None, **kw)


@pytest.mark.parametrize("case,qs,os", [(1, 8, None), (1, None, 8), (2, 4, 16), (3, 8, 8), (5, 1, 32), (7, 8, 8),
                                        (10, 2, 2), (14, 8, 8), (15, 16, 4), (16, 8, None), (17, 8, 8),
                                        (19, None, 8), (22, 8, 8)])
def test_attention_factors(bat, case, qs, os):
    seqs, Hq, H, D, fmt, page, kw = CASES[case]
    s = Setup(bat, seqs, Hq, H, D, fmt, page, seed=100 + case, qf=qs, of=os)
    s.check(s.call(**kw), **kw)


@pytest.mark.parametrize("seqs", [[(1, 400), (1, 33)], [(70, 400), (9, 33)]])
def test_attention_strided_q_and_rows_behind(bat, seqs):
    """q as a slice of a wider row; rows behind the last sequence stay as they were."""
    s = Setup(bat, seqs, 8, 2, 128, "mxfp8", 16, seed=5, q_pad=512, extra_rows=3)
    out = torch.full((s.T + 3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s.T + 3, 8), 7.0, device="cuda")
    s.call(out=out, lse=lse)
    s.check(out, lse)
    assert torch.all(out[s.T:] == 7.0) and torch.all(lse[s.T:] == 7.0)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attention_scale(bat, scale):
    for seqs in ([(1, 300)], [(90, 300)]):
        s = Setup(bat, seqs, 4, 2, 64, "mxfp8", 16, seed=6)
        lse = torch.empty(s.T, 4, device="cuda")
        s.check(s.call(scale=scale, lse=lse), lse, scale=scale)


@pytest.mark.parametrize("kv_scale", [1e-6, 1e5])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_attention_far_scales(bat, fmt, kv_scale):
    """Values far from 1: the products' range does not clip them."""
    for seqs in ([(1, 300)], [(90, 300)]):
        s = Setup(bat, seqs, 4, 2, 64, fmt, 16, seed=7, kv_scale=kv_scale)
        s.check(s.call(scale=0.125 / kv_scale), scale=0.125 / kv_scale)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_attention_large_scores(bat, fmt):
    """Scores of several hundred: the maximum is taken off before the exponential."""
    for seqs in ([(1, 500)], [(100, 500)]):
        s = Setup(bat, seqs, 4, 2, 128, fmt, 16, seed=8)
        lse = torch.empty(s.T, 4, device="cuda")
        s.check(s.call(scale=30.0, lse=lse), lse, scale=30.0)


def test_attention_bad_page_hides_tokens(bat):
    """A table entry outside the cache hides its page and sets the error word."""
    for seqs in ([(1, 200)], [(80, 200)]):
        s = Setup(bat, seqs, 4, 2, 64, "mxfp8", 16, seed=9)
        assert bat.bat_device_error() == 0
        s.table[0, 2] = s.slots  # far outside
        out = s.call()
        torch.cuda.synchronize()
        assert bat.bat_device_error() == 16
        assert torch.isfinite(out.float()).all()
        # the hidden page's 16 tokens are as if they were not there
        n = seqs[0][0]
        keep = torch.cat([torch.arange(0, 32), torch.arange(48, 200)]).cuda()
        q = s.q.double()
        for h in range(2):
            k, v = s.vals[0][0][keep, h], s.vals[1][0][keep, h]
            x = torch.einsum("gd,kd->gk", q[n - 1, 2 * h:2 * h + 2], k) * 64 ** -0.5
            want = torch.softmax(x, -1) @ v
            mag = torch.softmax(x, -1) @ v.abs()
            err = (out[n - 1, 2 * h:2 * h + 2].double() - want).abs()
            assert torch.all(err <= 2 * U * (mag + want.abs()) + 2 ** -12 * mag)


def test_attention_nan_only_where_seen(bat):
    """A stored NaN reaches the rows that see it and no other, whatever tile they share."""
    n, L = 100, 260
    s = Setup(bat, [(n, L), (1, 30)], 4, 2, 64, "mxfp8", 16, seed=10)
    ref = s.call()
    j = 200  # position 200 = new token 40: rows 40.. see it
    slot = int(s.table[0, j // 16]) * 16 + j % 16
    k8 = s.caches[0].codes.view(s.slots, 2, 64)
    v8 = s.caches[1].codes.view(s.slots, 2, 64)
    old = int(k8[slot, 0, 3])
    k8[slot, 0, 3] = 0x7F
    out = s.call().float()
    assert torch.isnan(out[40:100, 0:2]).all()
    assert torch.equal(out[:40], ref[:40].float()) and torch.equal(out[:, 2:], ref[:, 2:].float())
    assert torch.equal(out[100:], ref[100:].float())
    k8[slot, 0, 3] = old
    v8[slot, 1, 5] = 0xFF
    out = s.call().float()
    assert torch.isnan(out[40:100, 2:4, 5]).all()
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[40:100, 2:4, 5] = False
    assert torch.equal(out[rest], ref.float()[rest])


def test_attention_lengths_read_on_the_device(bat):
    """A captured call is replayed with other lengths, tables and queries."""
    a = Setup(bat, [(1, 2000), (1, 10), (1, 900)], 8, 2, 128, "mxfp8", 16, seed=11)
    ws = torch.empty(bat.bat_kv_attention_workspace_bytes(3, 8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    a.call(out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(out=out, workspace=ws)
    for lens in ([2000, 10, 900], [1, 10, 17], [1500, 0, 900], [33, 4, 5]):
        a.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        b = a.seqs
        a.seqs = [(1, n) for n in lens]
        vals = a.vals
        a.vals = [[None if v is None else v[:n] for v, n in zip(x, lens)] for x in vals]
        a.check(out)
        a.seqs, a.vals = b, vals


def test_attention_is_deterministic_and_streams(bat):
    """Same bits on every run, on another stream, and for two calls in flight."""
    for seqs in ([(1, 3000), (1, 17), (1, 1200)], [(200, 3000), (64, 64)]):
        s = Setup(bat, seqs, 8, 2, 128, "mxfp8", 16, seed=12)
        ref = s.call()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        outs = []
        for k in range(6):
            outs.append(s.call(stream=(s1, s2)[k & 1]))
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)


def test_attention_wrong_max_q_len_is_still_right(bat):
    s = Setup(bat, [(200, 500), (1, 3)], 8, 2, 64, "mxfp8", 16, seed=13)
    s.check(s.call(max_q_len=1))
    s = Setup(bat, [(1, 500), (1, 3)], 8, 2, 64, "mxfp8", 16, seed=14)
    s.check(s.call(max_q_len=4096))


def test_attention_clamps_lengths(bat):
    """A length past the table is clamped and reported; nothing outside is read."""
    s = Setup(bat, [(1, 64)], 4, 2, 64, "mxfp8", 16, seed=15, capacity=0)
    ref = s.call()
    s.kv_lens.fill_(1000)
    out = s.call()
    torch.cuda.synchronize()
    assert bat.bat_device_error() == 16
    assert torch.equal(out, ref)


def test_attention_batch_of_many_sequences(bat):
    """More sequences than a warp scans at once."""
    g = torch.Generator().manual_seed(3)
    seqs = [(int(torch.randint(0, 3, (1,), generator=g)), int(torch.randint(0, 200, (1,), generator=g)))
            for _ in range(77)]
    s = Setup(bat, seqs, 4, 2, 64, "mxfp8", 16, seed=16)
    s.check(s.call())


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("seqs", [[(1, 700)], [(40, 700)]])
def test_attention_tokens_of_very_different_size(bat, fmt, seqs):
    """Keys and values whose tokens differ by up to 2^24: the scales of a tile do not drown small ones."""
    s = Setup(bat, seqs, 4, 2, 128, fmt, 16, seed=17)
    g = torch.Generator().manual_seed(18)
    eyeA, eyeB = torch.eye(8).cuda(), torch.eye(4).repeat(4, 1, 1).cuda()
    L = seqs[0][1]
    j = torch.arange(L)
    slot = (s.table[0].cpu()[j // 16].long() * 16 + j % 16).cuda()
    for c in range(2):
        size = torch.exp2(torch.randint(-12, 13, (L, 1, 1), generator=g).float())
        x = (torch.randn(L, 2, 128, generator=g) * size).bfloat16().cuda()
        bat.bat_kv_quantize(x, eyeA, eyeB, slot, s.caches[c])
        s.vals[c][0] = bat.bat_kv_dequantize(s.caches[c], slot).double()
    for scale in (2.0 ** -14, 2.0 ** -8):
        s.check(s.call(scale=scale), scale=scale)


@pytest.mark.parametrize("seqs", [[(1, 300)], [(50, 300)]])
def test_attention_scales_at_any_address(bat, seqs):
    """Scale arrays that do not begin at a word."""
    s = Setup(bat, seqs, 4, 2, 128, "mxfp8", 16, seed=19)
    ref = s.call()
    for c in s.caches:
        wide = torch.zeros(c.scales.numel() + 8, dtype=torch.uint8, device="cuda")
        wide[1:1 + c.scales.numel()] = c.scales
        c.scales = wide[1:1 + c.scales.numel()]
    assert torch.equal(s.call(), ref)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attention_bad_q_stays_in_its_row(bat, value):
    for seqs in ([(1, 300), (1, 20)], [(50, 300), (7, 20)]):
        s = Setup(bat, seqs, 4, 2, 64, "mxfp8", 16, seed=20)
        ref = s.call()
        s.q[0, 1, 5] = value
        out = s.call()
        assert torch.isnan(out[0, 1]).all()
        keep = torch.ones(s.T, 4, dtype=torch.bool, device="cuda")
        keep[0, 1] = False
        assert torch.equal(out[keep], ref[keep])


def test_attention_many_chunks_batch(bat):
    """More sequences than a warp scans at once, on the tile kernel, with a window."""
    g = torch.Generator().manual_seed(5)
    seqs = [(int(torch.randint(0, 40, (1,), generator=g)), int(torch.randint(1, 400, (1,), generator=g)))
            for _ in range(50)]
    for kw in ({}, {"window": 50, "sinks": 2}):
        s = Setup(bat, seqs, 6, 2, 64, "mxfp4", 16, seed=21)
        s.check(s.call(**kw), **kw)


@pytest.mark.parametrize("kw", [{"window": 10 ** 9}, {"window": 10 ** 9, "sinks": 10 ** 9}, {"sinks": 5}, {"window": 3, "sinks": 10 ** 9}])
def test_attention_windows_without_effect(bat, kw):
    """Windows and sinks that hide nothing give the plain result's bits."""
    for seqs in ([(1, 300), (1, 20)], [(90, 300), (7, 20)]):
        s = Setup(bat, seqs, 4, 2, 64, "mxfp8", 16, seed=22)
        ref, out = s.call(), s.call(**kw)
        if kw.get("window") == 3:
            s.check(out)  # every token is a sink: the same values, numbered another way
        else:
            assert torch.equal(out, ref)


def test_attention_two_graphs_in_flight(bat):
    """Two captured calls with workspaces of their own, replayed together on two streams."""
    calls = []
    for k, seqs in enumerate(([(1, 2500), (1, 40)], [(120, 2500)])):
        s = Setup(bat, seqs, 8, 2, 128, "mxfp8", 16, seed=23 + k)
        ref = s.call()
        torch.cuda.synchronize()
        out = torch.empty_like(ref)
        ws = torch.empty(bat.bat_kv_attention_workspace_bytes(s.T, 8, 2, 128, seqs[0][0]), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.call(out=out, workspace=ws)
        calls.append((s, ref, out, ws, g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for _, _, out, _, _, _ in calls:
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for _, _, _, _, g, st in calls:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for _, ref, out, _, _, _ in calls:
            assert torch.equal(out, ref)


def test_attention_right_after_the_store(bat):
    """Store, attend, overwrite and attend again without a wait between: each call sees its own cache."""
    for n in (1, 60):
        s = Setup(bat, [(n, 400)], 8, 2, 128, "mxfp8", 16, seed=25)
        eyeA, eyeB = torch.eye(8).cuda(), torch.eye(4).repeat(4, 1, 1).cuda()
        j = torch.arange(400)
        slot = (s.table[0].cpu()[j // 16].long() * 16 + j % 16).cuda()
        g = torch.Generator().manual_seed(26)
        xs = [torch.randn(400, 2, 128, generator=g).bfloat16().cuda() for _ in range(6)]
        alone = []
        for x in xs:
            bat.bat_kv_quantize(x, eyeA, eyeB, slot, s.caches[0])
            bat.bat_kv_quantize(x, eyeA, eyeB, slot, s.caches[1])
            torch.cuda.synchronize()
            alone.append(s.call())
            torch.cuda.synchronize()
        for _ in range(5):
            got = []
            for x in xs:
                bat.bat_kv_quantize(x, eyeA, eyeB, slot, s.caches[0])
                bat.bat_kv_quantize(x, eyeA, eyeB, slot, s.caches[1])
                got.append(s.call())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, alone))
