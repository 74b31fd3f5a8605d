"""RMS norm into the quantizer: transformed values against 64 bits, codes and scales bit for
bit against the oracle quantizer fed with the kernel's own transformed values.

Bar of the transformed values, relative to the block's largest: y = h inv w (three fp32
roundings, the sum of K squares and its root: less than 2^-24 (log2 K + 8) for a tree
of fp32 sums) and the transform's 12 (up to 32) multiply-adds over sums of |x P| whose entries
stay within a few times the block's largest value: 1e-5 in all, the quantizer's own bar.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import formats
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bat():
    import w4a4_bit_gemm_b200 as m
    m.lib()
    return m


def _inputs(M, K, seed, residual=True, s=8):
    g = torch.Generator().manual_seed(seed)
    big = torch.where(torch.rand(K, generator=g) < 0.02, 50.0, 1.0)
    x = (torch.randn(M, K, generator=g) * big).bfloat16().cuda()
    r = (torch.randn(M, K, generator=g) * 2).bfloat16().cuda() if residual else None
    w = (1 + 0.3 * torch.randn(K, generator=g)).bfloat16().cuda()
    t = 32 // s
    A = (torch.eye(s) + 0.1 * torch.randn(s, s, generator=g)).cuda()
    B = (torch.eye(t) + 0.1 * torch.randn(K // 32, t, t, generator=g)).cuda()
    lo = (1 + 3 * torch.rand(K // 32, generator=g)).cuda()
    hi = (1 + 3 * torch.rand(K // 32, generator=g)).cuda()
    return x, r, w, A.contiguous(), B.contiguous(), lo, hi


def _check(bat, M, K, fmt, seed, residual=True, s=8, clip=True, xform=True, inplace=False, eps=1e-6):
    x, r, w, A, B, lo, hi = _inputs(M, K, seed, residual, s)
    y = torch.empty(M, K, dtype=torch.float32, device="cuda")
    h = x.double() + (r.double() if residual else 0.0)
    kw = dict(residual=r, eps=eps, fmt=fmt)
    if xform:
        kw.update(A=A, B=B)
    if clip:
        kw.update(g_lo=lo, g_hi=hi)
    q2, r2 = bat.bat_rmsnorm_quantize(x, w, **kw)  # without the trace
    out = r if inplace else None
    q, ro = bat.bat_rmsnorm_quantize(x, w, y_out=y, residual_out=out, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)
    if residual:
        want = h.float().bfloat16()  # x + r of two bf16 is exact in 64 bits; fp32 and bf16 round it in turn
        assert torch.equal(ro, want) and torch.equal(r2, want)
        if inplace:
            assert ro.data_ptr() == r.data_ptr()
    else:
        assert ro is None
    ref = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * w.double()
    nb = K // 32
    if xform:
        P = torch.stack([torch.kron(b.double(), A.double()) for b in B])
        ref = torch.einsum("mbk,bkn->mbn", ref.view(M, nb, 32), P)
    ref = ref.reshape(M, nb, 32)
    err = (y.double().view(M, nb, 32) - ref).abs().amax(2)
    assert torch.all(err <= 1e-5 * ref.abs().amax(2)), (err / ref.abs().amax(2).clamp(min=1e-300)).max()
    r_lo = bat.bat_clip_ratios(lo if clip else None, nb).cpu().numpy()
    r_hi = bat.bat_clip_ratios(hi if clip else None, nb).cpu().numpy()
    tiled = q.scales.cpu().numpy()
    scales = formats.untile_scales(tiled, M, nb)
    oc, os_, _ = oracle.quantize(y.cpu().numpy(), r_lo, r_hi, **({"fmt": "e4m3"} if fmt == "mxfp8" else {}))
    codes = q.codes.cpu().numpy()
    codes = codes.reshape(M, K) if fmt == "mxfp8" else formats.unpack_codes(codes.reshape(M, K // 2))
    assert np.array_equal(codes, oc) and np.array_equal(scales, os_)
    assert np.all(tiled[formats.padding_mask(M, nb)] == 0)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 4096), (16, 4096), (3, 96), (130, 160), (777, 2880), (400, 4096),
                                 (2, 8192), (350, 8192), (5, 12288), (33, 16384), (2, 16416), (3, 40960)])
def test_norm_shapes(bat, fmt, M, K):
    _check(bat, M, K, fmt, seed=M + K)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("kw", [dict(residual=False), dict(clip=False), dict(xform=False), dict(inplace=True),
                                dict(xform=False, clip=False, residual=False), dict(eps=0.1),
                                dict(s=1), dict(s=2), dict(s=4), dict(s=16), dict(s=32)])
@pytest.mark.parametrize("M,K", [(5, 416), (300, 4096), (2, 16480)])
def test_norm_options(bat, fmt, kw, M, K):
    _check(bat, M, K, fmt, seed=7, **kw)


def test_norm_zero_rows(bat):
    """An all-zero row: eps keeps the root finite, codes 0, scale byte 0."""
    x, r, w, A, B, lo, hi = _inputs(4, 256, 3)
    x[1] = 0
    r[1] = 0
    q, ro = bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r)
    assert torch.all(q.codes.view(4, 256)[1] == 0)
    assert np.all(formats.untile_scales(q.scales.cpu().numpy(), 4, 8)[1] == 0)
    assert torch.all(ro[1] == 0)


def test_norm_residual_out_without_residual_and_x_in_place(bat):
    x, r, w, A, B, lo, hi = _inputs(50, 512, 4)
    ro = torch.empty_like(x)
    q, got = bat.bat_rmsnorm_quantize(x, w, A, B, residual_out=ro)
    assert got is ro and torch.equal(ro, x)
    q1, r1 = bat.bat_rmsnorm_quantize(x, w, A, B, residual=r)
    q2, r2 = bat.bat_rmsnorm_quantize(x, w, A, B, residual=r, residual_out=x)  # over X
    assert torch.equal(q1.codes, q2.codes) and torch.equal(r1, x) and r2 is x


def test_norm_graph_and_streams(bat):
    x, r, w, A, B, lo, hi = _inputs(300, 4096, 5)
    q0, r0 = bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    q1, r1 = bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(q0.codes, q1.codes) and torch.equal(r0, r1)
    q2, r2 = bat.MXFP8.empty(300, 4096), torch.empty_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r, Xq=q2, residual_out=r2)
    q2.codes.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q0.codes, q2.codes) and torch.equal(q0.scales, q2.scales) and torch.equal(r0, r2)


def test_decoder_step(bat):
    """The run of operators around one decoder attention, as a user strings them together: norm into
    the quantizer, qkv product, K and V into the cache, attention with the head transforms
    undone, output product; against the same in 64 bits on the dequantized operands."""
    T, K, Hq, H, D, page = 150, 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(9)
    x, r, w, A, B, lo, hi = _inputs(T, K, 10)
    N = (Hq + 2 * H) * D
    Wqkv = (0.05 * torch.randn(N, K, generator=g)).bfloat16().cuda()
    Wq = bat.bat_prepare_weight(Wqkv, A, B)
    nb = D // 32
    Ak = (torch.eye(8) + 0.1 * torch.randn(8, 8, generator=g)).cuda()
    Bk = (torch.eye(4) + 0.1 * torch.randn(nb, 4, 4, generator=g)).cuda()
    iT = lambda m: torch.linalg.inv(m.double()).transpose(-1, -2).float().contiguous()
    inv = lambda m: torch.linalg.inv(m.double()).float().contiguous()
    Xq, res = bat.bat_rmsnorm_quantize(x, w, A, B, lo, hi, residual=r, fmt="mxfp4")
    qkv = bat.bat_mxfp4_gemm(Xq, Wq)
    heads = qkv.view(T, Hq + 2 * H, D)
    slots = torch.arange(T, device="cuda") + page
    kc, vc = (bat.KVCache.empty(page * 12, H, D, "mxfp8") for _ in range(2))
    bat.bat_kv_quantize(heads[:, Hq:Hq + H].contiguous(), Ak, Bk, slots, kc)
    bat.bat_kv_quantize(heads[:, Hq + H:].contiguous(), Ak, Bk, slots, vc)
    table = torch.arange(1, 11, dtype=torch.int32, device="cuda").view(1, 10)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    att = bat.bat_kv_attention(heads[:, :Hq], kc, vc, table, i32(T), i32(0, T), page, T,
                               q_factors=(iT(Ak), iT(Bk)), out_factors=(inv(Ak), inv(Bk)))
    Ao, Bo = torch.eye(8).cuda(), torch.eye(4).repeat(Hq * D // 32, 1, 1).cuda()
    Wo = bat.bat_prepare_weight((0.05 * torch.randn(K, Hq * D, generator=g)).bfloat16().cuda(), Ao, Bo)
    y = bat.bat_linear(att.view(T, Hq * D), Wo, Ao, Bo)
    torch.cuda.synchronize()
    assert y.shape == (T, K) and torch.isfinite(y.float()).all() and bat.bat_device_error() == 0
    # the transforms cancel: attention of the cache read back through the inverse factors
    k = bat.bat_kv_dequantize(kc, slots, inv(Ak), inv(Bk)).double()
    v = bat.bat_kv_dequantize(vc, slots, inv(Ak), inv(Bk)).double()
    q = heads[:, :Hq].double()
    k, v = (t.repeat_interleave(Hq // H, 1) for t in (k, v))
    s = torch.einsum("thd,khd->htk", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    p = torch.softmax(s, -1)
    want, mag = torch.einsum("htk,khd->thd", p, v), torch.einsum("htk,khd->thd", p, v.abs())
    # bf16 steps of the output, the weights and q' (its scores: 2^-8 sum |q'||k'| scale, less than
    # 2^-8 * 4 |s|max here), with a factor 2 for the transforms' norms
    tol = 2 * 2 ** -8 * (want.abs() + mag.amax(-1, keepdim=True) * (1 + 8 * s[s.isfinite()].abs().max()))
    assert torch.all((att.double() - want).abs() <= tol)
