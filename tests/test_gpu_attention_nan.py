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
