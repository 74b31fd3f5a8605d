"""Stored NaN in the attention calls: they reach the rows that see their token, in the channels that they are
in, and nothing else."""
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


def _codes_seen(c, marks):
    """`marks` [tokens][H][D] (bool): which outputs see one."""
    seen = torch.zeros(c.T, c.Hq, c.D, dtype=torch.bool)
    t0 = l0 = 0
    G = c.Hq // c.H
    for n, L in c.seqs:
        upto = marks[l0:l0 + L].to(torch.int32).cumsum(0) > 0
        for i in range(n):
            p = L - n + i
            if p >= 0:
                seen[t0 + i] = upto[p].repeat_interleave(G, 0)
        t0 += n
        l0 += L
    return seen


@pytest.mark.parametrize("D", [64, 128])
def test_nan_of_the_last_rows_before_a_short_sequence(bat, D):
    """Many NaN codes that only the last rows of a chunk see (their look-up is long), the next sequence's few rows
    right behind on the same SM."""
    seqs = [(64, 4000), (8, 3900)] * 30
    c = Case(bat, seqs, 8, 2, D, "mxfp8", seed=1)
    marks = torch.zeros(c.total, 2, D, dtype=torch.bool)
    l0 = 0
    for n, L in seqs:
        j = torch.arange(L - 24, L)
        marks[l0 + j, :, j % D] = True
        marks[l0 + j, :, (5 * j + 3) % D] = True
        l0 += L
    c.V.codes[marks] = 0
    ref, _ = c.call()
    c.V.codes[marks] = 0x7F
    out, _ = c.call()
    seen = _codes_seen(c, marks)
    assert torch.equal(torch.isnan(out), seen)
    assert torch.equal(out[~seen], ref[~seen])


SEQS = pytest.mark.parametrize("seqs", [[(1, 300), (1, 45)], [(1, 5000)], [(3, 300)], [(100, 260), (7, 40)]])
FMT = pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])


@FMT
@SEQS
@pytest.mark.parametrize("D", [64, 96, 256])
def test_nan_scale_of_v(bat, fmt, seqs, D):
    """A scale byte 255 in V: the block's channels of the rows that see it."""
    c = Case(bat, seqs, 4, 2, D, fmt, seed=2)
    L = seqs[0][1]
    c.V.scales[L - 40, 0, 1] = 255   # rows near the end, head 0
    c.V.scales[3, 1, 0] = 255        # all rows, head 1
    c.V.scales[L - 1, 1, 1] = 255    # the last row
    c.check()


@FMT
@SEQS
@pytest.mark.parametrize("D", [64, 128])
def test_nan_scale_of_k(bat, fmt, seqs, D):
    """A scale byte 255 in K: the whole of the rows that see it, their sum too."""
    c = Case(bat, seqs, 4, 2, D, fmt, seed=3)
    c.K.scales[seqs[0][1] - 40, 0, 1] = 255
    c.K.scales[seqs[0][1] - 1, 1, 0] = 255
    _, lse = c.check()
    assert torch.isnan(lse[seqs[0][0] - 1]).all()


@SEQS
def test_nan_codes(bat, seqs):
    c = Case(bat, seqs, 6, 2, 128, "mxfp8", seed=4)
    L = seqs[0][1]
    c.V.codes[L - 30, 0, 77] = 0x7F
    c.V.codes[10, 1, 5] = 0xFF
    c.V.codes[L - 1, 1, 127] = 0x7F
    c.K.codes[L - 2, 0, 3] = 0xFF
    c.check()


@FMT
@SEQS
def test_nan_outside_the_window(bat, fmt, seqs):
    c = Case(bat, seqs, 4, 2, 64, fmt, seed=5)
    c.V.scales[100, 0, 1] = 255
    c.K.scales[101, 1, 0] = 255
    c.check(window=50, sinks=2)


@FMT
@SEQS
def test_nan_beside_large_scales(bat, fmt, seqs):
    """NaN in tokens and blocks that go the rare ways."""
    c = Case(bat, seqs, 4, 2, 128, fmt, seed=6)
    L = seqs[0][1]
    c.V.shift((slice(0, None, 4), slice(None), 2), 60)
    c.V.scales[L - 33, 0, 1] = 255
    c.V.scales[L - 36, 0, 2] = 255
    c.K.shift((slice(7, None, 16), slice(None), 0), -60)
    c.K.scales[L - 34, 1, 1] = 255
    if fmt == "mxfp8":
        c.V.codes[L - 32, 1, 70] = 0x7F
        c.K.codes[7, 0, 1] = 0x7F
    c.check()
