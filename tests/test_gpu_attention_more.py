"""Attention calls at sizes and arguments beside the usual: every group size of the row kernel's variants, lengths
and starts that point outside, values near the ends of the range."""
from __future__ import annotations

import pytest
import torch

from attention_range import Case

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])


@pytest.fixture(scope="module")
def bat():
    import w4a4_bit_gemm_b200 as m
    m.lib()
    return m


@FMT
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 224, 256])
@pytest.mark.parametrize("group", [1, 5, 8, 9, 16, 17, 40])
def test_every_group_size(bat, fmt, D, group):
    """Up to 8 heads to a KV head, up to 16, and several units of them."""
    Case(bat, [(1, 650), (1, 1), (1, 131)], 2 * group, 2, D, fmt, seed=D + group).check()


@FMT
@pytest.mark.parametrize("D", [32, 96, 160, 256])
@pytest.mark.parametrize("group", [1, 3, 16, 40])
def test_every_group_size_in_chunks(bat, fmt, D, group):
    Case(bat, [(13, 300), (60, 200), (1, 77)], 2 * group, 2, D, fmt, seed=D + group).check()


@FMT
@pytest.mark.parametrize("seqs", [[(1, 300)], [(50, 300)]])
def test_values_near_the_range(bat, fmt, seqs):
    for by in (90, -40):
        c = Case(bat, seqs, 4, 2, 128, fmt, seed=1)
        c.V.shift(slice(None), by)
        c.check()
    # one value of V far above all others, at a weight of almost nothing and at a usual one
    c = Case(bat, seqs, 4, 2, 128, fmt, seed=2)
    c.V.shift((5, slice(None), 1), 90)
    c.check()


def _touched(c, out, lse, rows):
    rest = torch.ones(c.T, dtype=torch.bool)
    rest[rows] = False
    assert torch.all(out[rest] == 7.0) and torch.all(lse[rest] == 7.0)


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("starts", ["below", "behind", "descending"])
def test_starts_outside(bat, chunk, starts):
    """Starts below 0, behind the last token or descending: clamped, reported, nothing else written."""
    n = 40 if chunk else 1
    c = Case(bat, [(n, 300), (n, 200), (n, 100)], 4, 2, 64, "mxfp8", seed=3)
    good, gl = c.check()
    assert bat.bat_device_error() == 0
    if starts == "below":
        c.q_starts = [-5, n, 2 * n, 3 * n]
        rows = [slice(0, n), slice(n, 2 * n), slice(2 * n, 3 * n)]
    elif starts == "behind":
        c.q_starts = [0, n, 2 * n, 3 * n + 1000]
        rows = [slice(0, n), slice(n, 2 * n), slice(2 * n, 3 * n)]
    else:
        c.q_starts = [0, n, 0, 0]
        rows = [slice(0, n)]
    out, lse = c.call()
    assert bat.bat_device_error() == 16
    for r in rows:
        assert torch.equal(out[r], good[r]) and torch.equal(lse[r], gl[r])
    _touched(c, out, lse, torch.cat([torch.arange(c.T)[r] for r in rows]))
    assert bat.bat_device_error() == 0


@pytest.mark.parametrize("lens", [10 ** 6, 2 ** 31 - 1, -1, -2 ** 31])
@pytest.mark.parametrize("n", [1, 256])
def test_lengths_outside(bat, n, lens):
    """A length over the table's capacity counts as the capacity, one below 0 as 0; both are reported."""
    c = Case(bat, [(n, 512), (1, 300)], 16, 8, 128, "mxfp8", seed=4)
    c.table = c.table[:, :32].contiguous()  # 512 tokens of 16 a page
    good, gl = c.check()
    assert bat.bat_device_error() == 0
    c.kv_lens = [lens, 300]
    out, lse = c.call()
    assert bat.bat_device_error() == 16
    assert torch.equal(out[n:], good[n:]) and torch.equal(lse[n:], gl[n:])
    if lens > 0:
        assert torch.equal(out, good) and torch.equal(lse, gl)
    else:
        assert torch.all(out[:n] == 0) and torch.all(torch.isneginf(lse[:n]))


@pytest.mark.parametrize("seqs", [[(1, 200)], [(60, 200)]])
@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1])
def test_page_entries_outside(bat, seqs, entry):
    """A page that is not there hides its tokens, as if their scores were -inf."""
    c = Case(bat, seqs, 4, 2, 64, "mxfp4", seed=5)
    c.table[0, 5] = entry
    out, lse = c.call()
    assert bat.bat_device_error() == 16
    keep = torch.cat([torch.arange(0, 80), torch.arange(96, 200)])
    n = seqs[0][0]
    k, v = c.K.values(), c.V.values()
    for h in range(4):
        x = c.q[:, h].double() @ k[keep, h // 2].T * 64 ** -0.5
        x = x.masked_fill(keep[None] > torch.arange(200 - n, 200)[:, None], float("-inf"))
        p = torch.softmax(x, 1)
        # bars as in attention_range, with the scores' term at its largest here
        mag = p @ v[keep, h // 2].abs()
        assert torch.all((out[:, h].double() - p @ v[keep, h // 2]).abs() <= 2.0 ** -7 * mag)
        assert torch.all((lse[:, h].double() - torch.logsumexp(x, 1)).abs() <= 2.0 ** -12)
