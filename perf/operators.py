"""Operators of a decoder layer around the low-bit linear: attention over the paged
MXFP8 / MXFP4 cache, and the RMS norm that feeds the quantizer.

Every case is a dict of plain values; ``run`` computes it either in plain torch
(``own`` false) or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------ cases
# Attention: B sequences, the longest with n new tokens and L tokens in the cache (new ones
# among them); `ragged` spreads both over the batch. Pages of `page` tokens in any order.
# factors: the K and V paths carry head transforms, undone on q and on the output.


def _attn(name, B, n, L, **kw):
    c = {"op": "attention", "name": name, "B": B, "n": n, "L": L, "ragged": False, "Hq": 32, "Hkv": 8,
         "D": 128, "fmt": "mxfp8", "page": 64, "window": 0, "sinks": 0, "factors": False, "lse": False}
    c.update(kw)
    return c


def _norm(name, M, K, **kw):
    c = {"op": "norm", "name": name, "M": M, "K": K, "fmt": "mxfp8", "residual": True}
    c.update(kw)
    return c


def listed():
    return [
        # one user, one token: the latency of a chat's next token
        _attn("decode_one", 1, 1, 1000, page=16, lse=True),
        # a serving batch's step, contexts of all lengths, with the head transforms
        _attn("decode_batch", 16, 1, 4096, ragged=True, factors=True),
        # few users with very long contexts in the 4-bit cache
        _attn("decode_long_kv4", 8, 1, 65536, fmt="mxfp4"),
        # a large batch of a sliding-window model with narrow heads and seven of them to a group
        _attn("decode_window", 64, 1, 8192, ragged=True, Hq=28, Hkv=4, D=64, page=32, window=1024, sinks=4),
        # drafted tokens verified together
        _attn("verify_drafts", 8, 5, 2000, ragged=True, page=16),
        # a chunk of a long prompt over what the cache already has
        _attn("chunk_long", 1, 2048, 16384),
        # a mixed batch: prompts' ends and odd lengths, pages that end inside a tile, 4 bits
        _attn("chunk_ragged_kv4", 6, 777, 5000, ragged=True, fmt="mxfp4", page=24, factors=True),
        # prompts of a sliding-window model with sinks
        _attn("chunk_window", 2, 4096, 4500, window=1024, sinks=4, lse=True),
        # the norm before decode's qkv projection, 4-bit activations
        _norm("norm_decode", 16, 4096, fmt="mxfp4"),
        # an odd batch and width, first layer (no residual yet)
        _norm("norm_odd", 777, 2880, residual=False),
        # prefill before gate/up
        _norm("norm_prefill", 2048, 4096),
        # long prefill
        _norm("norm_long", 16384, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        if rng.random() < 0.35:
            fmt = rng.choice(["mxfp8", "mxfp8", "mxfp4"])
            c = _norm("", _log(rng, 1, 64 if fmt == "mxfp4" else 16384), 32 * _log(rng, 16, 384), fmt=fmt,
                      residual=rng.random() < 0.7)
        else:
            hkv = rng.choice([1, 2, 4, 5, 8])
            n = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
            c = _attn("", _log(rng, 1, 64), n, n + _log(rng, 1, 65536), ragged=rng.random() < 0.6, Hkv=hkv,
                      Hq=hkv * rng.choice([1, 3, 4, 7, 8]), D=rng.choice([64, 64, 96, 128, 128, 128, 256]),
                      fmt=rng.choice(["mxfp8", "mxfp4"]), page=rng.choice([1, 16, 24, 32, 64, 128]),
                      factors=rng.random() < 0.3)
            if rng.random() < 0.35:
                c["window"], c["sinks"] = _log(rng, 16, 4096), rng.choice([0, 1, 4, 100])
            c["lse"] = not c["factors"] and rng.random() < 0.3
            # what the plain form holds: scores, the gathered cache
            scores = c["B"] * c["Hq"] * c["n"] * c["L"]
            cache = c["B"] * c["L"] * c["Hkv"] * c["D"]
            if scores > 1.2e9 or cache > 5.5e8:
                continue
        del c["name"]
        if _cost(c) <= top:
            return c


# ------------------------------------------------------------------ shapes
def _lens(c):
    """New tokens and cached tokens of every sequence (host integers)."""
    n, kv = [], []
    for b in range(c["B"]):
        f = 1.0 if not c["ragged"] or b == 0 else ((b * 0.6180339887) % 1.0)
        nb = max(1, int(c["n"] * f))
        n.append(nb)
        kv.append(max(nb, int(c["L"] * (0.1 + 0.9 * f))))
    return np.array(n, dtype=np.int64), np.array(kv, dtype=np.int64)


def _pairs(c):
    """(visible pairs, cached tokens that some row sees), summed over the batch."""
    n, kv = _lens(c)
    pairs = seen = 0
    for nb, L in zip(n, kv):
        p = np.arange(L - nb, L, dtype=np.int64)
        lo = np.maximum(0, p - c["window"] + 1) if c["window"] else np.zeros_like(p)
        pairs += int((p + 1 - lo + np.minimum(lo, c["sinks"])).sum())
        seen += int(L - lo[0] + min(lo[0], c["sinks"]))
    return pairs, seen


def work(c):
    if c["op"] == "norm":
        e = c["M"] * c["K"]
        out = 1.0 if c["fmt"] == "mxfp8" else 0.5
        return {"bytes": e * (2 + (4 if c["residual"] else 0) + out + 1 / 32) + 2 * c["K"], "flops": e * 32.0}
    n, kv = _lens(c)
    pairs, seen = _pairs(c)
    row = c["D"] * (1 if c["fmt"] == "mxfp8" else 0.5) + c["D"] // 32
    return {"bytes": 2.0 * seen * c["Hkv"] * row + 4.0 * int(n.sum()) * c["Hq"] * c["D"] + 4.0 * int(kv.sum()) / c["page"],
            "flops": 4.0 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------ inputs
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _quantize(x, fmt):
    """Codes and scale bytes of the last axis in blocks of 32 (x is fp32)."""
    blk = x.unflatten(-1, (-1, 32))
    amax = blk.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 1 - (8 if fmt == "mxfp8" else 2)).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    v = torch.ldexp(blk, -e.unsqueeze(-1))
    if fmt == "mxfp8":
        codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8)
    else:
        # nearest of the grid, ties to the even code
        a = v.abs()
        code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
                + (a >= 3.5).int() + (a > 5.0).int())
        code = (code + 8 * torch.signbit(v).int()).flatten(-2).to(torch.uint8)
        codes = code[..., 0::2] | (code[..., 1::2] << 4)
    return codes.contiguous(), (e + 127).to(torch.uint8).contiguous()


def _factors(g, nb, dev):
    eye8, eye4 = torch.eye(8, device=dev), torch.eye(4, device=dev)
    A = eye8 + 0.1 * torch.randn(8, 8, generator=g, device=dev)
    B = eye4 + 0.1 * torch.randn(nb, 4, 4, generator=g, device=dev)
    return A.contiguous(), B.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c = case
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        # a residual stream with a few large channels, and the update of the block before
        big = torch.where(torch.rand(K, generator=g, device=dev) < 0.01,
                          30 + 70 * torch.rand(K, generator=g, device=dev), torch.ones(K, device=dev))
        x = (torch.randn(M, K, generator=g, device=dev) * (0.3 if c["residual"] else big)).bfloat16()
        r = (torch.randn(M, K, generator=g, device=dev) * big).bfloat16() if c["residual"] else None
        w = (1 + 0.2 * torch.randn(K, generator=g, device=dev)).bfloat16()
        A, B = _factors(g, K // 32, dev)
        lo = 1 + 3 * torch.rand(K // 32, generator=g, device=dev)
        hi = 1 + 3 * torch.rand(K // 32, generator=g, device=dev)
        # the E4M3 bytes of the E2M1 values of a byte's two codes
        grid = torch.tensor(_E2M1 + [-v for v in _E2M1], device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
        byte = torch.arange(256, device=dev)
        lut = torch.stack([grid[byte & 15], grid[byte >> 4]], 1).contiguous()
        return {"case": c, "x": x, "r": r, "w": w, "A": A, "B": B, "lo": lo, "hi": hi, "lut": lut}
    n, kv = _lens(c)
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    pages = -(-kv // page)
    maxp = int(pages.max())
    pool = int(pages.sum()) + 3
    order = torch.randperm(pool, generator=g, device=dev)
    first = np.concatenate([[0], np.cumsum(pages)[:-1]])
    idx = first[:, None] + np.minimum(np.arange(maxp)[None, :], pages[:, None] - 1)
    table = order[torch.from_numpy(idx).to(dev)].to(torch.int32).contiguous()
    slots = pool * page
    big = torch.where(torch.rand(Hkv, D, generator=g, device=dev) < 0.03, 4.0, 1.0)
    kc, ks = _quantize(torch.randn(slots, Hkv, D, generator=g, device=dev) * big, c["fmt"])
    vc, vs = _quantize(torch.randn(slots, Hkv, D, generator=g, device=dev), c["fmt"])
    q = (1.5 * torch.randn(int(n.sum()), Hq, D, generator=g, device=dev)).bfloat16()
    s = {"case": c, "q": q, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "slots": slots, "table": table,
         "kv_lens": torch.from_numpy(kv).to(dev).to(torch.int32),
         "q_starts": torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(dev).to(torch.int32),
         "max_q": int(n.max()), "qf": None, "of": None,
         "lut": torch.tensor(_E2M1 + [-v for v in _E2M1], device=dev)}
    if c["factors"]:
        s["qf"] = _factors(g, D // 32, dev)
        s["of"] = _factors(g, D // 32, dev)
    return s


# ------------------------------------------------------------------ plain forms
def _block_transform(x, A, B):
    """x_b (B_b (x) A) for every 32-channel block of the last axis."""
    nb = B.shape[0]
    x = x.unflatten(-1, (nb, 4, 8))
    return torch.einsum("...bip,bij,pq->...bjq", x, B, A).flatten(-3)


def _values(codes, scales, fmt, lut):
    """Stored values of cache rows in fp32."""
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


def _plain_attention(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    kv, qs = s["kv_lens"].long(), s["q_starts"].long()
    n = qs[1:] - qs[:-1]
    Lm, Nm = s["table"].shape[1] * page, s["max_q"]
    j = torch.arange(Lm, device=kv.device)
    i = torch.arange(Nm, device=kv.device)
    rows = (qs[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)          # [B, N]
    pos = (kv - n)[:, None] + i
    slot = s["table"].long()[:, j // page] * page + j % page           # [B, L]
    see = (j <= pos[..., None]) & (i[:, None] < n[:, None, None])      # [B, N, L]
    if c["window"]:
        see &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    q = s["q"].float()
    if s["qf"] is not None:
        q = _block_transform(q, *s["qf"])
    q = q[rows].unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G N, D]
    hrow = s["kc"].shape[-1]
    k = _values(s["kc"].view(-1, Hkv, hrow)[slot], s["ks"].view(-1, Hkv, D // 32)[slot], c["fmt"], s["lut"])
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).unflatten(2, (G, Nm))         # [B, Hkv, G, N, L]
    del k
    x.mul_(1 / math.sqrt(D)).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    v = _values(s["vc"].view(-1, Hkv, hrow)[slot], s["vs"].view(-1, Hkv, D // 32)[slot], c["fmt"], s["lut"])
    o = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (G, Nm))
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    if s["of"] is not None:
        o = _block_transform(o, *s["of"])
    real = i < n[:, None]
    out = {"out": o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].bfloat16()}   # [T, Hq, D]
    if c["lse"]:
        out["lse"] = (l.log() + m).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)[real]
    return out


def _tiled_scales(sb, M, nb):
    """Scale bytes [M][nb] in the GEMM's tiled order, padding 0."""
    mt, bt = -(-M // 128), -(-nb // 4)
    t = torch.zeros(mt * 128, bt * 4, dtype=torch.uint8, device=sb.device)
    t[:M, :nb] = sb
    return t.view(mt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).contiguous().flatten()


def _plain_norm(s):
    c = s["case"]
    M, K, nb = c["M"], c["K"], c["K"] // 32
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    y = _block_transform(y, s["A"], s["B"]).unflatten(-1, (nb, 32))
    lo = torch.sigmoid(s["lo"].double()).float() * y.amin(-1)
    hi = torch.sigmoid(s["hi"].double()).float() * y.amax(-1)
    y = torch.minimum(torch.maximum(y, lo[..., None]), hi[..., None])
    amax = y.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - (8 if c["fmt"] == "mxfp8" else 2)
    e = torch.where(amax > 0, e.clamp(min=-127), torch.full_like(e, -127))
    v = torch.ldexp(y, -e[..., None])
    if c["fmt"] == "mxfp8":
        el = v.clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        a = v.abs()
        k = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
             + (a >= 3.5).int() + (a > 5.0).int())
        el = torch.copysign(torch.tensor(_E2M1, device=v.device)[k.long()], v).to(torch.float8_e4m3fn)
    out = {"elements": el.reshape(M, K),
           "scales": _tiled_scales((e + 127).to(torch.uint8), M, nb).view(torch.float8_e8m0fnu)}
    if s["r"] is not None:
        out["residual"] = h.bfloat16()
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_norm(s) if c["op"] == "norm" else _plain_attention(s)
    import w4a4_bit_gemm_b200 as bat
    if c["op"] == "norm":
        xq, res = bat.bat_rmsnorm_quantize(s["x"], s["w"], s["A"], s["B"], s["lo"], s["hi"], residual=s["r"],
                                           eps=1e-6, fmt=c["fmt"])
        if c["fmt"] == "mxfp8":
            el = xq.codes.view(torch.float8_e4m3fn).view(c["M"], c["K"])
        else:
            el = s["lut"][xq.codes.int()].view(torch.float8_e4m3fn).view(c["M"], c["K"])
        out = {"elements": el, "scales": xq.scales.view(torch.float8_e8m0fnu)}
        if res is not None:
            out["residual"] = res
        return out
    kc = bat.KVCache(s["kc"].view(-1), s["ks"].view(-1), s["slots"], c["Hkv"], c["D"], c["fmt"])
    vc = bat.KVCache(s["vc"].view(-1), s["vs"].view(-1), s["slots"], c["Hkv"], c["D"], c["fmt"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device) if c["lse"] else None
    out = {"out": bat.bat_kv_attention(s["q"], kc, vc, s["table"], s["kv_lens"], s["q_starts"], c["page"], s["max_q"],
                                       window=c["window"], sinks=c["sinks"], q_factors=s["qf"],
                                       out_factors=s["of"], lse=lse)}
    if lse is not None:
        out["lse"] = lse
    return out


# ------------------------------------------------------------------ 64 bits
def _dense_blocks(A, B):
    """[nb][32][32] fp64 matrices kron(B_b, A)."""
    return torch.stack([torch.kron(b.double(), A.double()) for b in B])


def exact(case, seed):
    s, c = prepare(case, seed), case
    return _exact_norm(s, c) if c["op"] == "norm" else _exact_attention(s, c)


def _exact_norm(s, c):
    M, K = c["M"], c["K"]
    P = _dense_blocks(s["A"], s["B"])
    r_lo, r_hi = 1 / (1 + torch.exp(-s["lo"].double())), 1 / (1 + torch.exp(-s["hi"].double()))
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=s["x"].device)
    els, sbs, hs = [], [], []
    for at in range(0, M, 2048):
        h = s["x"][at:at + 2048].double()
        if s["r"] is not None:
            h = h + s["r"][at:at + 2048].double()
            hs.append(h)
        y = h / torch.sqrt((h ** 2).sum(1, keepdim=True) / K + 1e-6) * s["w"].double()
        y = torch.matmul(y.view(-1, K // 32, 1, 32), P).squeeze(2)
        a, b = r_lo[:, None] * y.amin(2, True), r_hi[:, None] * y.amax(2, True)
        y = y.clamp(a, b)
        top = y.abs().amax(2, True)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -130)))
        e = torch.where(torch.exp2(e) > top, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
        e = (e - (8 if c["fmt"] == "mxfp8" else 2)).clamp(min=-127)
        v = y / torch.exp2(e)
        if c["fmt"] == "mxfp8":
            # three fraction bits, exponents from -6 up, nearest with ties to even
            mag = v.abs()
            step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
            el = torch.sign(v) * torch.clamp(torch.round(mag / step) * step, max=448.0)
        else:
            # nearest of the grid; on a tie the neighbour with the even code
            mag = v.abs().clamp(max=6.0)
            up = torch.searchsorted(grid, mag.contiguous()).clamp(1, 7)
            d = (grid[up] - mag) - (mag - grid[up - 1])
            take = (d < 0) | ((d == 0) & (up % 2 == 0))
            el = torch.sign(v) * torch.where(take, grid[up], grid[up - 1])
        els.append(el.reshape(-1, K))
        sbs.append(torch.exp2(e.squeeze(2)))
    nb, sc = K // 32, torch.cat(sbs)
    out = torch.full((-(-M // 128), -(-nb // 4), 32, 4, 4), 2.0 ** -127, dtype=torch.float64, device=sc.device)
    m, b = torch.arange(M, device=sc.device)[:, None], torch.arange(nb, device=sc.device)[None, :]
    out[m // 128, b // 4, m % 32, m % 128 // 32, b % 4] = sc
    res = {"elements": torch.cat(els), "scales": out.flatten()}
    if hs:
        res["residual"] = torch.cat(hs)
    return res


def _exact_attention(s, c):
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    G, dev = Hq // Hkv, s["q"].device
    n, kv = _lens(c)
    pairs = Hq * sum(int(a) * int(b) for a, b in zip(n, kv))
    if pairs * D > 4e11 or len(n) * Hkv > 2000:
        return None
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=dev)

    def stored(codes, scales, slots, h):
        x = codes.view(-1, Hkv, codes.shape[-1])[slots, h]
        if c["fmt"] == "mxfp4":
            x = torch.stack([x & 15, x // 16], -1).flatten(1).long()
            x = grid[x % 8] * (1 - 2 * (x // 8))
        else:
            x = x.view(torch.float8_e4m3fn).double()
        e = scales.view(-1, Hkv, D // 32)[slots, h].double() - 127
        return x * torch.pow(2.0, e).repeat_interleave(32, 1)

    q = s["q"].double()
    if s["qf"] is not None:
        P = _dense_blocks(*s["qf"])
        q = torch.cat([q[..., 32 * b:32 * b + 32] @ P[b] for b in range(D // 32)], -1)
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, (nb, L) in enumerate(zip(n.tolist(), kv.tolist())):
        j = torch.arange(L, device=dev)
        slots = s["table"][b].long()[torch.div(j, page, rounding_mode="floor")] * page + j % page
        for h in range(Hkv):
            k, v = stored(s["kc"], s["ks"], slots, h), stored(s["vc"], s["vs"], slots, h)
            for i0 in range(0, nb, 512):
                i1 = min(nb, i0 + 512)
                p = torch.arange(L - nb + i0, L - nb + i1, device=dev)[:, None]
                hide = j > p
                if c["window"]:
                    hide = hide | ((j <= p - c["window"]) & (j >= c["sinks"]))
                t = slice(at + i0, at + i1)
                x = torch.einsum("tgd,kd->tgk", q[t, h * G:(h + 1) * G], k) * D ** -0.5
                x = x.masked_fill(hide[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[t, h * G:(h + 1) * G] = z
                out[t, h * G:(h + 1) * G] = torch.exp(x - z[..., None]) @ v
        at += nb
    if s["of"] is not None:
        P = _dense_blocks(*s["of"])
        out = torch.cat([out[..., 32 * b:32 * b + 32] @ P[b] for b in range(D // 32)], -1)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
