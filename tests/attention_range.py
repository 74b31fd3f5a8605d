"""Attention cases whose stored codes and scale bytes are written directly, and their values and error
bars in 64 bits: for tests of sizes that a quantized Gaussian does not have.

Bars, per output channel d of a row, from the arithmetic (p_j the softmax weights, v_j the values):
  * each weight is rounded once for the product: u p_j |v_jd|, u half a step of its format relative to
    the value: 2^-11 (single tokens), 2^-8 (chunks);
  * a score is off by at most e_j = 2^-22 sqrt(D) scale sum_d |q_d k_jd| + 2^-22 (fp32 sums of D exact
    products, the subtraction of the maximum, the exponential), which changes its weight by a factor
    within exp(+-2 e_j) and the weights' sum in proportion;
  * fp32 sums over the tokens: 2^-16 sum_j p_j |v_jd| covers 2^-24 times a few hundred partial sums;
  * weights below 2^-110 of the row's largest (single tokens: times the token's V scale), and products
    below 2^-94, may be lost;
  * the output is rounded once to bf16: 2^-8 |out|.
q is bf16 and goes to f16 by a power of two a row, exactly for channels within 2^-28 of the row's
largest; q below are far inside that.
"""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


class Stored:
    """Codes [tokens][H][D] (one a byte) and scale bytes [tokens][H][D/32] of one sequence after another."""

    def __init__(self, L, H, D, fmt, g):
        self.fmt = fmt
        if fmt == "mxfp8":
            # magnitudes up to 448 with the usual mix of exponents; no NaN
            x = (100 * torch.randn(L, H, D, generator=g)).clamp(-448, 448)
            self.codes = x.to(torch.float8_e4m3fn).view(torch.uint8).clone()
        else:
            self.codes = torch.randint(0, 16, (L, H, D), generator=g, dtype=torch.uint8)
        # values of about 1
        self.scales = torch.full((L, H, D // 32), 127 - (7 if fmt == "mxfp8" else 1), dtype=torch.int64)

    def shift(self, index, by):
        self.scales[index] += by

    def values(self):
        if self.fmt == "mxfp8":
            v = self.codes.view(torch.float8_e4m3fn).double()
        else:
            v = E2M1[(self.codes & 7).long()] * (1.0 - 2.0 * (self.codes >> 3).double())
        s = torch.where(self.scales == 255, math.nan, torch.pow(2.0, self.scales.double() - 127))
        return v * s.repeat_interleave(32, 2)

    def write(self, cache, slot):
        codes = self.codes if self.fmt == "mxfp8" else self.codes[..., 0::2] | (self.codes[..., 1::2] << 4)
        H = self.codes.shape[1]
        cache.codes.view(cache.num_slots, H, -1)[slot] = codes.to(cache.codes.device)
        cache.scales.view(cache.num_slots, H, -1)[slot] = self.scales.to(torch.uint8).to(cache.scales.device)


class Case:
    def __init__(self, bat, seqs, Hq, H, D, fmt, seed=0, page=16, q=None):
        g = torch.Generator().manual_seed(seed)
        self.bat, self.seqs, self.Hq, self.H, self.D, self.fmt, self.page = bat, seqs, Hq, H, D, fmt, page
        self.T, self.total = sum(n for n, _ in seqs), sum(L for _, L in seqs)
        self.K, self.V = Stored(self.total, H, D, fmt, g), Stored(self.total, H, D, fmt, g)
        self.q = (torch.randn(self.T, Hq, D, generator=g) if q is None else q).bfloat16()
        pages = [max(1, -(-L // page)) for _, L in seqs]
        # chunks: a table with room for many tokens, so that the call goes to the tile kernel
        self.max_q = max(n for n, _ in seqs)
        room = (1 << 20) // page if self.max_q > 1 else max(pages)
        self.slots = (sum(pages) + 2) * page
        order = torch.randperm(sum(pages) + 2, generator=g)
        self.table = torch.full((len(seqs), room), 2 ** 30, dtype=torch.int32)
        slot, at = [], 0
        for b, ((_, L), n) in enumerate(zip(seqs, pages)):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
            j = torch.arange(L)
            slot.append(self.table[b, j // page].long() * page + j % page)
        self.slot = torch.cat(slot)
        self.kv_lens = [L for _, L in seqs]
        self.q_starts = [0]
        for n, _ in seqs:
            self.q_starts.append(self.q_starts[-1] + n)

    def call(self, **kw):
        bat = self.bat
        dev = torch.device("cuda")
        caches = []
        for st in (self.K, self.V):
            c = bat.KVCache.empty(self.slots, self.H, self.D, self.fmt)
            c.codes.fill_(0x7F)  # rows of no sequence: NaN
            c.scales.fill_(255)
            st.write(c, self.slot.to(dev))
            caches.append(c)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
        lse = torch.full((self.T, self.Hq), 7.0, device=dev)
        out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=dev)
        bat.bat_kv_attention(self.q.to(dev), *caches, self.table.to(dev), i32(self.kv_lens), i32(self.q_starts),
                             self.page, self.max_q, out=out, lse=lse, **kw)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def reference(self, window=0, sinks=0, scale=None, row_kernel=None):
        """out, bar, lse in 64 bits (CPU): rows that see a NaN are NaN where they see it."""
        scale = self.D ** -0.5 if scale is None else scale
        row_kernel = self.max_q == 1 if row_kernel is None else row_kernel
        u = 2.0 ** -11 if row_kernel else 2.0 ** -8
        G, D = self.Hq // self.H, self.D
        k_all, v_all = self.K.values(), self.V.values()
        out = torch.zeros(self.T, self.Hq, D, dtype=torch.float64)
        bar, lse = torch.zeros_like(out), torch.full((self.T, self.Hq), -math.inf, dtype=torch.float64)
        self.lse_bar = torch.zeros_like(lse)
        t0 = l0 = 0
        for n, L in self.seqs:
            pos, j = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
            see = j <= pos
            if window:
                see = see & ((j > pos - window) | (j < sinks))
            for h in range(self.Hq):
                k, v = k_all[l0:l0 + L, h // G], v_all[l0:l0 + L, h // G]
                q = self.q[t0:t0 + n, h].double()
                x = (q @ k.T * scale).masked_fill(~see, -math.inf)
                a = (q.abs() @ k.abs().T * abs(scale)).masked_fill(~see, 0.0)
                m = x.amax(1, keepdim=True)
                none = ~see.any(1)  # rows that see nothing: out 0, lse -inf
                m[none] = 0.0
                w = torch.exp(x - m)
                z = w.sum(1, keepdim=True)
                p = torch.where(none[:, None], 0.0, w / z)
                e = torch.expm1(2 * (a * 2.0 ** -22 * math.sqrt(D) + 2.0 ** -22).clamp(max=300.0))
                e = torch.where(p > 0, e, 0.0)
                # (a value that a row does not see takes no part, a NaN neither)
                vv = torch.where(see[:, :, None], v[None], 0.0)
                o = torch.einsum("tk,tkd->td", p, vv)
                mag = torch.einsum("tk,tkd->td", p, vv.abs())
                off = torch.einsum("tk,tkd->td", p * e, vv.abs())
                big = (p[:, :, None] * vv.abs()).nan_to_num(0.0).amax((1, 2))[:, None]
                b = mag * (u + 2.0 ** -16) + off + o.abs() * (p * e).sum(1, keepdim=True) + L * (2.0 ** -94 + big * 2.0 ** -110)
                if not row_kernel:
                    lost = torch.where(p < 2.0 ** -110 * p.amax(1, keepdim=True), p, 0.0)
                    b = b + torch.einsum("tk,tkd->td", lost, vv.abs().nan_to_num(0.0))
                out[t0:t0 + n, h] = o
                bar[t0:t0 + n, h] = b * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs()
                lse[t0:t0 + n, h] = (m + torch.log(z)).squeeze(1)
                # the scores' errors, and fp32's of the maximum, the sum and the logarithm
                self.lse_bar[t0:t0 + n, h] = (p * e).sum(1) + 2.0 ** -20 + 2.0 ** -21 * lse[t0:t0 + n, h].abs()
            t0 += n
            l0 += L
        return out, bar, lse

    def check(self, **kw):
        out, lse = self.call(**kw)
        ref, bar, z = self.reference(**kw)
        nan = torch.isnan(ref)
        got = out.double()
        assert torch.equal(torch.isnan(got), nan), "NaN where the row sees none, or none where it sees one"
        err = (got - ref).abs()
        bad = ~nan & ~(err <= bar)
        assert not bad.any(), (torch.argwhere(bad)[:4].tolist(), int(bad.sum()),
                               float((err / bar)[bad].max()), float((err / ref.abs())[bad].max()))
        off = torch.where(torch.isneginf(z) & torch.isneginf(lse), 0.0, (lse.double() - z).abs())
        assert torch.equal(torch.isnan(lse), torch.isnan(z))
        assert not (~torch.isnan(z) & ~(off <= self.lse_bar)).any(), float((off / self.lse_bar).nan_to_num(0.0).max())
        return out, lse
