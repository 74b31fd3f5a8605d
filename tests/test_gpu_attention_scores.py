"""Attention with very large scores: the largest one takes all of the weight, and the output is its value."""
from __future__ import annotations

import pytest
import torch

from attention_range import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bat():
    import w4a4_bit_gemm_b200 as m
    m.lib()
    return m


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 70)], [(1, 6000)], [(40, 300), (7, 70)]])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("size", [8, 14, 18, 22, 28, 34, 50, 80])
def test_large_scores(bat, fmt, seqs, sign, size):
    """Scores of about +-2^size, one token's above all others by far more than fp32's step: out is that
    token's value, to the rounding of one weight (2^-11, 2^-8 in chunks) and of the output (2^-8)."""
    T = sum(n for n, _ in seqs)
    g = torch.Generator().manual_seed(size)
    c = Case(bat, seqs, 6, 2, 128, fmt, seed=size, q=sign * (0.5 + torch.rand(T, 6, 128, generator=g)))
    # every key along one direction, sizes 1 to 1.5 (2 to 4 in KV4), but for two tokens
    lo, hi = (0x38, 0x3C) if fmt == "mxfp8" else (4, 6)
    c.K.codes[:] = torch.randint(lo, hi, c.K.codes.shape[:2] + (1,), generator=g, dtype=torch.uint8)
    c.K.scales[:] = 127 + size - 4
    l0 = 0
    for _, L in seqs:
        # positive scores: the largest key wins; negative: the smallest. A later equal one shares the weight.
        win = (hi + 8 if fmt == "mxfp8" else 7) if sign > 0 else (lo - 16 if fmt == "mxfp8" else 1)
        c.K.codes[l0 + 11] = win
        c.V.shift((slice(l0, l0 + L, 3), 0, 1), -9)
        l0 += L
    out, lse = c.call()
    v = c.V.values()
    t0 = l0 = 0
    u = 2.0 ** -8 + (2.0 ** -11 if c.max_q == 1 else 2.0 ** -8)
    for n, L in seqs:
        want = v[l0 + 11].repeat_interleave(3, 0)[None]
        assert torch.isfinite(lse[t0:t0 + n]).all()
        assert torch.all((out[t0:t0 + n].double() - want).abs() <= u * want.abs() + 2.0 ** -90), \
            float(((out[t0:t0 + n].double() - want).abs() / want.abs().clamp(min=1e-9)).max())
        # the log sum: the winner's score
        k = c.K.values()[l0 + 11].repeat_interleave(3, 0)
        x = (c.q[t0:t0 + n].double() * k[None]).sum(-1) * 128 ** -0.5
        assert torch.all((lse[t0:t0 + n].double() - x).abs() <= 2.0 ** -19 * x.abs())
        t0 += n
        l0 += L


@pytest.mark.parametrize("seqs", [[(1, 300)], [(40, 300)]])
@pytest.mark.parametrize("size", [8, 20, 34, 60])
def test_equal_large_scores(bat, seqs, size):
    """Two tokens with the same key share the weight."""
    T = seqs[0][0]
    g = torch.Generator().manual_seed(3)
    c = Case(bat, seqs, 4, 2, 64, "mxfp8", seed=1, q=0.5 + torch.rand(T, 4, 64, generator=g))
    c.K.scales[:] = 127 + size - 8
    c.K.codes[:] = 0x30
    c.K.codes[5] = c.K.codes[201] = 0x50
    out, _ = c.call()
    v = c.V.values()
    want = ((v[5] + v[201]) / 2).repeat_interleave(2, 0)[None]
    mag = ((v[5].abs() + v[201].abs()) / 2).repeat_interleave(2, 0)[None]
    assert torch.all((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -8 * mag)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("seqs", [[(1, 300)], [(1, 6000)], [(40, 300)], [(100, 6000)]])
@pytest.mark.parametrize("steps", [(46, 95), (47, 100), (60, 100), (39, 39)])
def test_weights_that_wait_for_a_larger_one(bat, fmt, seqs, steps):
    """Scores that rise in steps from token to token: the weights of before are scaled down by far and still count
    where the largest one's value is zero."""
    n, L = seqs[0]
    first = L - n
    c = Case(bat, seqs, 2, 1, 64, fmt, seed=4, q=torch.ones(n, 2, 64))
    one, big = (0x38, 0x40) if fmt == "mxfp8" else (2, 4)  # 1 and 2
    c.K.codes[:] = 0
    c.K.scales[:] = 127
    # 64 channels of 1 times 1 / 8: a key of one block's first channels gives the score; log2 units: / ln 2
    at = [first // 4, first // 256 * 128 + 100, first - 1]  # (the second behind others of its chunk)
    score = [-8.0, -8.0 + steps[0], -8.0 + steps[0] + steps[1]]
    for j, s in zip(at, score):
        want = round(s * 0.6931 * 8)  # sum of the key's channels
        size = abs(want) // 64 + 1
        e = max(0, size.bit_length())
        c.K.codes[j, 0] = one | ((0x80 if fmt == "mxfp8" else 8) if want < 0 else 0)
        c.K.codes[j, 0, abs(want) * 64 // (64 * 2 ** e):] = 0
        c.K.scales[j] = 127 + e
    c.V.codes[at[2], 0, 20:] = 0
    c.V.shift(at[1], 50)
    c.check()
