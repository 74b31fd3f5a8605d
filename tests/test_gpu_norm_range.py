"""RMS norm into the quantizer where values are not finite or the instances that the usual shapes do not reach: the
codes and scale bytes of the oracle, which gives a block that holds a value that is not finite the scale byte 255 (NaN)
and codes 0."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import formats
from test_gpu_norm import _check, _inputs

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])


@pytest.fixture(scope="module")
def bat():
    import w4a4_bit_gemm_b200 as m
    m.lib()
    return m


def _codes(q, M, K, fmt):
    c = q.codes.cpu().numpy()
    c = c.reshape(M, K) if fmt == "mxfp8" else formats.unpack_codes(c.reshape(M, K // 2))
    return c, formats.untile_scales(q.scales.cpu().numpy(), M, K // 32)


@FMT
@pytest.mark.parametrize("kw", [dict(xform=False), dict(s=1), dict(s=4), dict(s=16), dict(s=32), dict(s=8)])
@pytest.mark.parametrize("M,K", [(3, 8224), (2, 12288), (5, 16384)])
def test_norm_two_vectors_a_thread(bat, fmt, kw, M, K):
    """8192 < K <= 16384 with any split and with no transform."""
    _check(bat, M, K, fmt, seed=M + K, **kw)


@FMT
@pytest.mark.parametrize("kw", [dict(s=2), dict(s=16), dict(xform=False)])
@pytest.mark.parametrize("M,K", [(700, 512), (1, 64)])
def test_norm_many_short_rows(bat, fmt, kw, M, K):
    _check(bat, M, K, fmt, seed=M + K, **kw)


@FMT
@pytest.mark.parametrize("xform", [True, False])
@pytest.mark.parametrize("clip", [True, False])
@pytest.mark.parametrize("K", [256, 4096, 12288, 20480])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 3e38, 1e25])
def test_norm_rows_that_are_not_finite(bat, fmt, xform, clip, K, value):
    """A NaN, an infinity or a sum of squares beyond fp32 makes its row NaN and leaves the others alone."""
    M = 6
    x, r, w, A, B, lo, hi = _inputs(M, K, K)
    kw = dict(residual=r, fmt=fmt)
    if xform:
        kw.update(A=A, B=B)
    if clip:
        kw.update(g_lo=lo, g_hi=hi)
    q0, _ = bat.bat_rmsnorm_quantize(x, w, **kw)
    x[2, K // 2 + 5] = value
    x[4, 3] = value
    q, ro = bat.bat_rmsnorm_quantize(x, w, **kw)
    c0, s0 = _codes(q0, M, K, fmt)
    c, s = _codes(q, M, K, fmt)
    for m in range(M):
        if m in (2, 4):
            assert np.all(s[m] == 255) and np.all(c[m] == 0)
        else:
            assert np.array_equal(c[m], c0[m]) and np.array_equal(s[m], s0[m])
    h = (x.double() + r.double()).float().bfloat16()
    assert torch.equal(torch.isnan(ro), torch.isnan(h)) and torch.equal(ro.nan_to_num(7.0), h.nan_to_num(7.0))


@FMT
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_norm_weight_that_is_not_finite(bat, fmt, value):
    """Without a transform a weight reaches its own channel: its block is NaN in every row, the others are not."""
    x, r, w, _, _, lo, hi = _inputs(5, 512, 9)
    w[70] = value
    q, _ = bat.bat_rmsnorm_quantize(x, w, g_lo=lo, g_hi=hi, residual=r, fmt=fmt)
    c, s = _codes(q, 5, 512, fmt)
    bad = np.arange(16) == 70 // 32
    assert np.all((s == 255) == bad[None]) and np.all(c[:, 64:96] == 0)


@FMT
def test_norm_zero_rows_without_eps(bat, fmt):
    """0 / 0: NaN; beside rows that are not zero."""
    x, r, w, A, B, lo, hi = _inputs(4, 256, 3)
    x[1] = 0
    r[1] = 0
    y = torch.empty(4, 256, device="cuda")
    q, _ = bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r, eps=0.0, fmt=fmt, y_out=y)
    c, s = _codes(q, 4, 256, fmt)
    rl, rh = (bat.bat_clip_ratios(g, 8).cpu().numpy() for g in (lo, hi))
    oc, os_, bad = oracle.quantize(y.cpu().numpy(), rl, rh, **({"fmt": "e4m3"} if fmt == "mxfp8" else {}))
    assert bad == 8 and np.array_equal(c, oc) and np.array_equal(s, os_) and np.all(s[1] == 255)


@pytest.mark.parametrize("fmt,M", [("mxfp4", 6), ("mxfp4", 200), ("mxfp4", 600), ("mxfp8", 6), ("mxfp8", 200)])
def test_norm_nan_rows_through_the_product(bat, fmt, M):
    """The product after it gives NaN for such a row, and the other rows' bits do not change."""
    K, N = 512, 512
    x, r, w, A, B, lo, hi = _inputs(M, K, 11)
    g = torch.Generator().manual_seed(12)
    Wq = bat.bat_prepare_weight((0.05 * torch.randn(N, K, generator=g)).bfloat16().cuda(), A, B)
    run = bat.bat_mxfp4_gemm if fmt == "mxfp4" else bat.bat_w4a8_gemm
    ref = run(bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r, fmt=fmt)[0], Wq)
    x[3, 100] = float("nan")
    x[M - 1, 100] = float("inf")
    y = run(bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r, fmt=fmt)[0], Wq)
    torch.cuda.synchronize()
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[3] = rows[M - 1] = False
    assert torch.isnan(y[~rows]).all() and torch.equal(y[rows], ref[rows])
