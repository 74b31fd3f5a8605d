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
