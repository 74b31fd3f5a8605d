"""Attention over caches whose blocks and tokens differ far in size: what a row sees decides its
result, to the bits that the header promises, in single tokens and in chunks."""
from __future__ import annotations

import math

import pytest
import torch

from attention_range import Case

pytestmark = pytest.mark.gpu

FMT = pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
SEQS = pytest.mark.parametrize("seqs", [[(1, 300), (1, 45)], [(1, 9000)], [(40, 300), (5, 45)]])


@pytest.fixture(scope="module")
def bat():
    import w4a4_bit_gemm_b200 as m
    m.lib()
    return m


# ------------------------------------------------------------------ values that differ in size
@FMT
@SEQS
@pytest.mark.parametrize("apart", [12, 20, 30])
def test_v_blocks_of_a_token_apart(bat, fmt, seqs, apart):
    """Every token's blocks of V differ by powers of two: each block of the output keeps its bits."""
    c = Case(bat, seqs, 8, 2, 128, fmt, seed=apart)
    for b in range(4):
        c.V.shift((slice(None), 0, b), -apart * b // 3)
        c.V.shift((slice(None), 1, b), -apart * ((b * 2 + 1) % 4) // 3)
    c.check()


@FMT
@SEQS
@pytest.mark.parametrize("up", [12, 26])
def test_v_one_large_block_of_one_token(bat, fmt, seqs, up):
    """One block of one token far above everything else: the other blocks do not notice."""
    c = Case(bat, seqs, 6, 2, 96, fmt, seed=100 + up)
    c.V.shift((7, slice(None), 1), up)
    c.check()


@FMT
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("Hq", [2, 24])
def test_v_blocks_apart_other_heads(bat, fmt, D, Hq):
    c = Case(bat, [(1, 700)], Hq, 2, D, fmt, seed=D + Hq)
    c.V.shift((slice(None), slice(None), 1), -22)
    c.V.shift((slice(0, None, 3), slice(None), 0), 9)
    c.check()


@FMT
@SEQS
@pytest.mark.parametrize("score", [12.0, 25.0, 50.0])
def test_long_tail_beside_a_dominant_token(bat, fmt, seqs, score):
    """A token far above the others in weight holds zeros in some channels: there the output is the sum of
    the others' small weights, which count with all their bits."""
    H, D = 2, 128
    T = sum(n for n, _ in seqs)
    g = torch.Generator().manual_seed(1)
    q = 0.5 + torch.rand(T, 4, D, generator=g)  # all of one sign: one key is near all of them
    c = Case(bat, seqs, 4, H, D, fmt, seed=2, q=q)
    one = 0x70 if fmt == "mxfp8" else 6  # 128 and 4
    c.K.codes[3] = one
    # codes of 2^7 (2^2) times the scale give about score / (sqrt(D) sum q / D) each
    e = round(math.log2(score / (math.sqrt(D) * 1.0))) - (7 if fmt == "mxfp8" else 2)
    c.K.scales[3] = 127 + e
    c.V.codes[3, :, 40:100] = 0
    c.check()


@FMT
@SEQS
def test_v_tiny_and_large_scales(bat, fmt, seqs):
    """All values far below or above 1: outputs follow them."""
    for by in (-100, -60, 30):
        c = Case(bat, seqs, 4, 2, 64, fmt, seed=3)
        c.V.shift(slice(None), by)
        if by == -100 and seqs[0][0] > 1:
            continue  # (chunks hold products in units of 2^-32 of fp32's range: see the header)
        c.check()

# ------------------------------------------------------------------ keys that differ in size
def _same_rows(bat, fmt, seqs, change, rows, D=128, **kw):
    """`change`s the keys of tokens that `rows` do not see: their bits stay."""
    c = Case(bat, seqs, 8, 2, D, fmt, seed=4)
    ref, rl = c.check(**kw)
    change(c.K)
    out, lse = c.call(**kw)
    assert torch.equal(out[rows], ref[rows]) and torch.equal(lse[rows], rl[rows])


@FMT
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("up", [14, 24, 40, 120])
def test_k_of_a_later_token(bat, fmt, D, up):
    """The last new token's key is far larger: the rows before it do not see it."""
    def change(K):
        K.scales[259] += up
    _same_rows(bat, fmt, [(100, 260)], change, slice(0, 99), D)


@FMT
@pytest.mark.parametrize("up", [24, 120])
def test_k_of_a_token_before_the_window(bat, fmt, up):
    def change(K):
        K.scales[170] += up
    # row i at position 160 + i sees 170 from i = 10 to 10 + 49
    _same_rows(bat, fmt, [(100, 260)], change, slice(60, 100), window=50, sinks=3)


@FMT
@SEQS
@pytest.mark.parametrize("up", [18, 26, 60])
def test_k_of_a_token_far_below_the_others_weight(bat, fmt, seqs, up):
    """A key far larger than its neighbours, against the rows' direction: its weight is 0 and the
    neighbours' scores count."""
    T = sum(n for n, _ in seqs)
    g = torch.Generator().manual_seed(5)
    c = Case(bat, seqs, 4, 2, 128, fmt, seed=6, q=0.2 + torch.rand(T, 4, 128, generator=g))
    c.K.codes[20] = 0x80 | 0x70 if fmt == "mxfp8" else 8 | 6
    c.K.scales[20] += up
    c.check()


@FMT
@SEQS
@pytest.mark.parametrize("up", [17, 30])
def test_k_blocks_of_a_token_apart(bat, fmt, seqs, up):
    """The first block of every key is far larger and meets zeros in q: the others decide."""
    T = sum(n for n, _ in seqs)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(T, 8, 128, generator=g)
    q[..., :32] = 0
    c = Case(bat, seqs, 8, 2, 128, fmt, seed=8, q=q)
    c.K.shift((slice(None), slice(None), 0), up)
    c.check()


@FMT
def test_k_zero_blocks(bat, fmt):
    """Blocks of zeros (scale byte 0, as the store writes them) beside ordinary ones."""
    c = Case(bat, [(60, 300)], 4, 2, 128, fmt, seed=9)
    for st in (c.K, c.V):
        st.codes[:, 0, 96:] = 0
        st.scales[:, 0, 3] = 0
        st.codes[5:90, 1] = 0
        st.scales[5:90, 1] = 0
    c.check()



# ------------------------------------------------------------------ V's largest scales
@FMT
@SEQS
@pytest.mark.parametrize("by", [36, 42, 60, 70])
def test_v_scales_above_the_usual(bat, fmt, seqs, by):
    """The same answer from single tokens and from chunks for large stored values."""
    c = Case(bat, seqs, 4, 2, 64, fmt, seed=10)
    c.V.shift(slice(None), by)
    c.check()
    c = Case(bat, seqs, 4, 2, 64, fmt, seed=11)
    c.V.shift((slice(2, None, 5), 1, 1), by)
    c.check()


@FMT
@pytest.mark.parametrize("apart", range(13, 32))
def test_v_block_far_below_in_the_largest_token(bat, fmt, apart):
    """Blocks far below in the one token that sets the weights' reference, the others' scales around its least."""
    c = Case(bat, [(1, 200), (1, 9)], 4, 2, 96, fmt, seed=apart)
    c.V.shift((5, slice(None), 1), apart)
    c.V.shift((204, 0, 2), apart)
    c.check(scale=0.0)
    c.check()
