"""Host-side checks of bat_kv_attention and bat_rmsnorm_quantize, without a GPU: the C-ABI refuses bad
arguments before any CUDA call, the binding refuses bad tensors before the library is called,
and the workspace sizes are those of the documented parts."""
from __future__ import annotations

import ctypes

import pytest
import torch

import w4a4_bit_gemm_b200 as bat

from test_binding_host import _RecordingLib


@pytest.fixture(scope="module")
def L():
    from w4a4_bit_gemm_b200 import build
    build.build()
    return bat.lib()


PTR = 0x7F0000000000


def _cache(**kw):
    f = dict(codes=PTR + 0x10000, scales=PTR + 0x20000, num_slots=64, H=2, D=64, fmt=0)
    f.update(kw)
    return bat.KVCacheStruct(*[f[k] for k in ("codes", "scales", "num_slots", "H", "D", "fmt")])


def _attention(L, K=None, V=None, **kw):
    a = dict(q=PTR, T=4, Hq=8, q_stride=8 * 64, table=PTR + 4, B=1, max_pages=4, page_size=16, kv=PTR + 8, qs=PTR + 12,
             max_q=1, scale=0.125, window=0, sinks=0, Aq=None, sq=8, Bq=None, Ao=None, so=8, Bo=None, out=PTR + 64,
             lse=None, ws=PTR + 0x40000, n=1 << 40)
    a.update(kw)
    K = _cache() if K is None else K
    V = _cache() if V is None else V
    return L.bat_kv_attention(a["q"], a["T"], a["Hq"], a["q_stride"], ctypes.byref(K), ctypes.byref(V), a["table"], a["B"],
                              a["max_pages"], a["page_size"], a["kv"], a["qs"], a["max_q"], a["scale"], a["window"],
                              a["sinks"], a["Aq"], a["sq"], a["Bq"], a["Ao"], a["so"], a["Bo"], a["out"], a["lse"], a["ws"],
                              a["n"], None)


INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 6, 7


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(kv=None), INVALID), (dict(qs=None), INVALID),
    (dict(out=None), INVALID), (dict(T=0), INVALID), (dict(Hq=0), INVALID), (dict(B=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(max_q=0), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(Aq=PTR), INVALID), (dict(Bo=PTR), INVALID), (dict(Aq=PTR, Bq=PTR, sq=3), UNSUPPORTED),
    (dict(Ao=PTR, Bo=PTR, so=64), UNSUPPORTED), (dict(Hq=7, q_stride=7 * 64), SHAPE), (dict(q_stride=8 * 64 - 8), SHAPE),
    (dict(q_stride=8 * 64 + 4), SHAPE), (dict(T=1 << 28), SHAPE), (dict(page_size=1 << 31), SHAPE),
    (dict(max_pages=1 << 31), SHAPE), (dict(q=PTR + 2), ALIGN), (dict(out=PTR + 8), ALIGN), (dict(table=PTR + 2), ALIGN),
    (dict(lse=PTR + 2), ALIGN), (dict(ws=PTR + 128), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=1024), WORKSPACE),
])
def test_attention_arguments(L, kw, status):
    assert _attention(L, **kw) == status


@pytest.mark.parametrize("cache,status", [
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(num_slots=0), INVALID), (dict(fmt=2), INVALID),
    (dict(D=48), SHAPE), (dict(D=288), SHAPE), (dict(codes=PTR + 8), ALIGN), (dict(num_slots=1 << 30), SHAPE),
])
def test_attention_caches(L, cache, status):
    assert _attention(L, K=_cache(**cache), V=_cache(**cache)) == status


def test_attention_caches_disagree(L):
    assert _attention(L, V=_cache(H=4)) == SHAPE
    assert _attention(L, V=_cache(num_slots=65)) == SHAPE
    assert _attention(L, V=_cache(fmt=1)) == UNSUPPORTED


def test_attention_workspace_sizes(L):
    up = lambda v: (v + 255) // 256 * 256
    size = bat.bat_kv_attention_workspace_bytes
    # single tokens: two parts of 8 (16 for more than 8 heads to a KV head, up to 128 channels)
    # rows for each of 592 CTAs, their maxima and sums, 48 bytes a CTA's mark
    parts = lambda ctas, rows, D: up(2 * ctas * rows * D * 4) + up(2 * ctas * rows * 8) + up(ctas * 40)
    for T, Hq, H, D, rows in ((1, 32, 8, 128, 8), (64, 28, 4, 64, 8), (3, 24, 2, 128, 16), (3, 24, 2, 256, 8)):
        assert size(T, Hq, H, D, 1) == parts(592, rows, D)
    # chunks: two parts of 256 rows for each of 160 CTAs, and q in 16 bits with a factor a row
    assert size(2048, 32, 8, 128, 2048) == parts(160, 256, 128) + up(2048 * 32 * 128 * 2) + up(2048 * 32 * 4)
    assert size(300, 4, 2, 192, 300) == parts(160, 128, 192) + up(300 * 4 * 192 * 2) + up(300 * 4 * 4)
    for bad in ((0, 8, 2, 64, 1), (4, 7, 2, 64, 1), (4, 8, 2, 48, 1), (4, 8, 2, 288, 1), (4, 8, 2, 64, 0), (1 << 28, 8, 2, 64, 1)):
        assert size(*bad) == 0


def _norm(L, **kw):
    Xq = kw.pop("Xq", bat.MXFP4Struct(PTR + 0x1000, PTR + 0x2000, 4, 64))
    a = dict(X=PTR, r=None, w=PTR + 0x100, M=4, K=64, eps=1e-6, A=PTR, s=8, B=PTR, lo=None, hi=None, fmt=0, ro=None, y=None)
    a.update(kw)
    return L.bat_rmsnorm_quantize(a["X"], a["r"], a["w"], a["M"], a["K"], a["eps"], a["A"], a["s"], a["B"], a["lo"], a["hi"],
                                  a["fmt"], ctypes.byref(Xq), a["ro"], a["y"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(w=None), INVALID), (dict(A=None), INVALID), (dict(lo=PTR), INVALID), (dict(M=0), INVALID),
    (dict(K=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(fmt=5), INVALID),
    (dict(s=5), UNSUPPORTED), (dict(K=48), SHAPE), (dict(M=5), SHAPE), (dict(K=262144 + 32), SHAPE), (dict(X=PTR + 2), ALIGN),
    (dict(r=PTR + 8), ALIGN), (dict(w=PTR + 2), ALIGN), (dict(ro=PTR + 4), ALIGN), (dict(y=PTR + 4), ALIGN),
    (dict(lo=PTR + 2, hi=PTR), ALIGN),
])
def test_norm_arguments(L, kw, status):
    assert _norm(L, **kw) == status


# ---------------------------------------------------------------- the binding
@pytest.fixture
def rec(monkeypatch):
    class Lib(_RecordingLib):
        SIZE = _RecordingLib.SIZE | {"bat_kv_attention_workspace_bytes"}
    r = Lib(bat.lib())
    monkeypatch.setattr(bat, "_lib", r)
    monkeypatch.setattr(bat, "_DEVICE_TYPE", "cpu")
    monkeypatch.setattr(bat, "_stream", lambda s: None)
    return r


def _call(q=None, fmt="mxfp8", **kw):
    D = 64
    a = dict(kcache=bat.KVCache.empty(64, 2, D, fmt, device="cpu"), vcache=bat.KVCache.empty(64, 2, D, fmt, device="cpu"),
             page_table=torch.zeros(2, 4, dtype=torch.int32), kv_lens=torch.zeros(2, dtype=torch.int32),
             q_starts=torch.zeros(3, dtype=torch.int32), page_size=16, max_q_len=1)
    a.update(kw)
    q = torch.zeros(4, 8, D, dtype=torch.bfloat16) if q is None else q
    return bat.bat_kv_attention(q, **a)


def test_attention_binding_reaches_the_library(rec):
    out = _call()
    assert out.shape == (4, 8, 64) and out.dtype == torch.bfloat16
    wide = torch.zeros(4, 12 * 64, dtype=torch.bfloat16)
    _call(q=wide[:, :512].unflatten(1, (8, 64)), lse=torch.empty(4, 8), window=8, sinks=1,
          q_factors=(torch.zeros(8, 8), torch.zeros(2, 4, 4)), out_factors=(torch.zeros(4, 4), torch.zeros(2, 8, 8)))
    assert rec.calls == ["bat_kv_attention"] * 2


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(4, 8, 64)), dict(q=torch.zeros(4, 512, dtype=torch.bfloat16)),
    dict(q=torch.zeros(8, 4, 64, dtype=torch.bfloat16).transpose(0, 1)),
    dict(q=torch.zeros(4, 8, 128, dtype=torch.bfloat16)[..., ::2]), dict(page_table=torch.zeros(2, 4, dtype=torch.int64)),
    dict(page_table=torch.zeros(8, dtype=torch.int32)), dict(page_table=torch.zeros(4, 2, dtype=torch.int32).t()),
    dict(kv_lens=torch.zeros(3, dtype=torch.int32)), dict(kv_lens=torch.zeros(2, dtype=torch.int64)),
    dict(q_starts=torch.zeros(2, dtype=torch.int32)), dict(lse=torch.zeros(4, 7)), dict(out=torch.zeros(4, 8, 64)),
    dict(out=torch.zeros(4, 8, 32, dtype=torch.bfloat16)), dict(workspace=torch.zeros(64)),
    dict(q_factors=(torch.zeros(8, 8), torch.zeros(3, 4, 4))), dict(out_factors=(torch.zeros(8, 4), torch.zeros(2, 4, 4))),
    dict(vcache=bat.KVCache.empty(64, 4, 64, "mxfp8", device="cpu")),
    dict(vcache=bat.KVCache.empty(32, 2, 64, "mxfp8", device="cpu")),
    dict(kcache=bat.KVCache(torch.zeros(8, dtype=torch.uint8), torch.zeros(64 * 4, dtype=torch.uint8), 64, 2, 64, "mxfp8")),
    dict(kcache=bat.KVCache(torch.zeros(64 * 128, dtype=torch.uint8), torch.zeros(8, dtype=torch.uint8), 64, 2, 64, "mxfp8")),
    dict(kcache=bat.KVCache(torch.zeros(64 * 128, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8), 64, 2, 64, "fp8")),
])
def test_attention_binding_refuses(rec, kw):
    with pytest.raises((ValueError, TypeError)):
        _call(**kw)
    assert rec.calls == []


def test_norm_binding(rec):
    X, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    A, B, g = torch.zeros(8, 8), torch.zeros(2, 4, 4), torch.zeros(2)
    q, r = bat.bat_rmsnorm_quantize(X, w, A, B, g, g, residual=X.clone())
    assert isinstance(q, bat.MXFP8) and r.shape == X.shape and q.codes.numel() == 256 and q.scales.numel() == 512
    q, r = bat.bat_rmsnorm_quantize(X, w, fmt="mxfp4")
    assert isinstance(q, bat.MXFP4) and r is None and q.codes.numel() == 128
    bat.bat_rmsnorm_quantize(X, w, torch.zeros(4, 4), torch.zeros(2, 8, 8), residual=X, residual_out=X)
    assert rec.calls == ["bat_rmsnorm_quantize"] * 3
    bad = [dict(weight=torch.zeros(64)), dict(weight=w[:32]), dict(A=A), dict(A=A, B=B[:1]), dict(g_lo=g), dict(g_lo=g, g_hi=g[:1]),
           dict(residual=X[:2]), dict(residual=X.float()), dict(fmt="fp8"), dict(Xq=bat.MXFP4.empty(4, 64, "cpu")),
           dict(Xq=bat.MXFP8(torch.zeros(8, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)),
           dict(residual_out=X[:2]), dict(y_out=torch.zeros(4, 32))]
    for kw in bad:
        a = dict(weight=w)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            bat.bat_rmsnorm_quantize(X, **a)
    for x in (X.float(), X[:, ::2], X[0]):
        with pytest.raises((ValueError, TypeError)):
            bat.bat_rmsnorm_quantize(x, w)
    assert len(rec.calls) == 3
