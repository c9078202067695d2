"""The paged cache and its attention in 64 bits, from the definitions in include/ep.h.

``Seqs`` makes a cache, its tables and the sequences' tokens; ``attention`` gives the
output with a bound of what fp32 arithmetic and 16-bit probabilities may do to it.
"""
from __future__ import annotations

import torch

from tests import layer_ref as ref

F64, U, BF16 = ref.F64, ref.U, ref.BF16


def rotate(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """fp64 rows [T, heads, D] by angles [T, R/2], each product and sum rounded to fp32
    (a product of two fp32 is exact in 64 bits, and so is the sum up to its own rounding)."""
    R = 2 * cos.shape[1]
    half = torch.arange(R // 2)
    ia, ib = (2 * half, 2 * half + 1) if interleaved else (half, half + R // 2)
    f = lambda v: v.float().to(F64)  # noqa: E731
    c, s = cos[:, None].to(F64), sin[:, None].to(F64)
    y = x.clone()
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = f(f(a * c) - f(b * s))
    y[..., ib] = f(f(b * c) + f(a * s))
    return y


def in_8_bits(x: torch.Tensor):
    """(E4M3 values, E8M0 bytes) of fp64 rows that are fp32 numbers: the row is the group."""
    floor = torch.tensor(1e-4, dtype=torch.float32).to(F64)
    s = (torch.maximum(x.abs().amax(-1), floor) / 448).float().to(F64)
    m, e = torch.frexp(s)
    e = torch.where(m == 0.5, e - 1, e)
    return ref.e4m3(x * torch.exp2(-e.to(F64))[..., None]), (e + 127).to(torch.uint8)


class Seqs:
    """B sequences of the given lengths and new tokens, over a shuffled paged cache.

    layout: "heads" (pages stored by head), "rows" (by row), "slice" (a part of a larger
    pool, by row).  Unused rows and pages hold NaN.  On the CPU; cuda() gives the handles.
    """

    def __init__(self, lens, new=None, Hq=4, Hkv=2, D=128, page=16, quant="none", layout="heads",
                 seed=0, extra_cols=1, spread=1.0, spare=3, gap=0, tail=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.new = g, list(lens), list(new) if new is not None else None
        self.Hq, self.Hkv, self.D, self.page, self.quant = Hq, Hkv, D, page, quant
        self.layout = layout
        B = len(self.lens)
        used = [-(-L // page) for L in self.lens]
        P = max(used + [1]) + extra_cols
        self.pages = sum(used) + spare
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((B, P), -7, dtype=torch.int32)  # never to be read there
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        n = self.new if self.new is not None else [1] * B
        self.starts = [gap]  # rows before the first sequence and behind the last: no one's
        for m in n:
            self.starts.append(self.starts[-1] + m)
        self.T = self.starts[-1] + tail if self.new is not None else B
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q = (spread * rand(self.T, Hq, D)).bfloat16()
        k, v = rand(self.pages, page, Hkv, D), rand(self.pages, page, Hkv, D)
        live = torch.zeros((self.pages, page), dtype=torch.bool)
        for b, L in enumerate(self.lens):
            for e in range(used[b]):
                live[self.table[b, e], :min(page, L - e * page)] = True
        self.live = live
        if quant == "none":
            self.k, self.v = k.bfloat16(), v.bfloat16()
            self.k[~live], self.v[~live] = float("nan"), float("nan")
            self.ks = self.vs = None
            self.kval, self.vval = self.k.to(F64), self.v.to(F64)
        else:
            self.k, self.ks, self.kval = self._fp8(k)
            self.v, self.vs, self.vval = self._fp8(v)

    def _fp8(self, x):
        q, e = in_8_bits(x.to(F64))
        byte = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
        byte[~self.live] = 0x7F
        e[~self.live] = 255
        val = torch.ldexp(ref.decode(byte), e[..., None].int() - 127)
        return byte, e.transpose(1, 2).contiguous(), val

    def _strided(self, x):
        x = x.cuda()
        if self.layout == "heads":
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if self.layout == "slice":
            pool = torch.zeros((x.shape[0] + 2, x.shape[1], x.shape[2] + 3, x.shape[3] + 16),
                               dtype=x.dtype, device="cuda")
            part = pool[1:-1, :, 2:-1, :x.shape[3]]
            part.copy_(x)
            return part
        return x.contiguous()

    def cuda(self):
        from combine_expert_histogram_gb300 import binding as ep

        scales = () if self.quant == "none" else (self.ks.cuda(), self.vs.cuda())
        cache = ep.KvCache(self._strided(self.k), self._strided(self.v), self.quant, *scales)
        start = torch.tensor(self.starts, dtype=torch.int32).cuda() if self.new is not None else None
        seqs = ep.new_kv_seqs(self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                              start)
        return cache, seqs, self.q.cuda()

    def rows(self, b, h):
        """Keys and values [len, D] of sequence b, head h."""
        L = self.lens[b]
        p = self.table[b, :-(-L // self.page)].long() if L else torch.zeros(0, dtype=torch.long)
        return (self.kval[p, :, h].reshape(-1, self.D)[:L], self.vval[p, :, h].reshape(-1, self.D)[:L])

    def attention(self, scale=None, window=0, sinks=0, device="cpu"):
        """(out, noise, lse, noise of lse) [T, Hq, ...]; rows without an owner are NaN.

        A logit is a sum of D products in fp32, by a unit that may cut off instead of
        rounding (2 U a step), times the scale: off by 2 (D + 4) U scale sum |q k|, and 2^-28
        of the row's largest |q| where q is held in fp16.  Its probability is then off by
        that, 4 roundings of the exponent's argument, the exponential's 2^-22, and 2^-8
        of itself for its rounding to 16 bits (in the numerator only), 2^-30 of the largest
        where it is held in fp16.  Sums of n terms in fp32: 2 n U of the terms' magnitudes,
        where n = 256 covers the chain of one tile's terms, tiles and parts being added
        with one rounding each.
        """
        D, G = self.D, self.Hq // self.Hkv
        scale = D ** -0.5 if scale is None else scale
        nan = float("nan")
        out = torch.full((self.T, self.Hq, D), nan, dtype=F64)
        noise, lse = torch.zeros_like(out), torch.full((self.T, self.Hq), nan, dtype=F64)
        noise_l = torch.zeros_like(lse)
        for b, L in enumerate(self.lens):
            t0, t1 = (self.starts[b], self.starts[b + 1]) if self.new is not None else (b, b + 1)
            n = t1 - t0
            i = torch.arange(L - n, L, device=device)[:, None]
            j = torch.arange(L, device=device)[None, :]
            seen = j <= i
            if window:
                seen = seen & ((i - j < window) | (j < sinks))
            for h in range(self.Hkv):
                k, v = (x.to(device) for x in self.rows(b, h))
                if L == 0 or n == 0:
                    out[t0:t1, h * G:(h + 1) * G] = 0.0
                    lse[t0:t1, h * G:(h + 1) * G] = float("-inf")
                    continue
                for g in range(h * G, (h + 1) * G):
                    q = self.q[t0:t1, g].to(F64).to(device)
                    o, e, ls, el = _rows(q, k, v, seen, scale, D)
                    out[t0:t1, g], noise[t0:t1, g] = o.cpu(), e.cpu()
                    lse[t0:t1, g], noise_l[t0:t1, g] = ls.cpu(), el.cpu()
        return out, noise, lse, noise_l

    def owned(self):
        own = torch.ones(self.T, dtype=torch.bool)
        if self.new is not None:
            own[:self.starts[0]] = False
            own[self.starts[-1]:] = False
        return own


def _rows(q, k, v, seen, scale, D):
    s = (q @ k.T * scale).masked_fill(~seen, float("-inf"))
    m = s.amax(1, keepdim=True)
    none = (m == float("-inf"))[:, 0]
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(1, keepdim=True)
    safe = torch.where(none[:, None], 1.0, total)
    off = 2 * (D + 4) * U * scale * (q.abs() @ k.abs().T)
    off = off + scale * 2.0 ** -28 * q.abs().amax(1, keepdim=True) * k.abs().sum(1)[None]
    off = off + 4 * U * (torch.where(seen, s, 0.0).abs() + m.abs()) + 2.0 ** -22
    n = s.shape[1]
    chain = 2 * U * (min(n, 256) + n / 64 + 64)
    v0 = torch.where(seen.any(0)[:, None], v, 0.0)
    o = p @ v0 / safe
    mag = p @ v0.abs() / safe
    e_num = ((p * (off + BF16)) @ v0.abs()) / safe + chain * mag
    e_num = e_num + 2.0 ** -30 * (seen.to(F64) @ v0.abs()) / safe
    e_den = (p * off).sum(1, keepdim=True) / safe + chain
    noise = (e_num + o.abs() * e_den) * 1.05
    lse = torch.where(none, torch.full_like(total[:, 0], float("-inf")), m[:, 0] + torch.log(safe[:, 0]))
    # the logarithm itself: 2^-22 and a rounding of the sum
    e_lse = 1.05 * (e_den[:, 0] + 2.0 ** -22) + 4 * U * (m[:, 0].abs() + torch.log(safe[:, 0]).abs())
    return o, noise, lse, e_lse


def close(s: Seqs, out: torch.Tensor, lse=None, **kw):
    """out (and lse) of a call are the formula's, rows without an owner aside."""
    want, noise, want_l, noise_l = s.attention(**kw)
    own = s.owned()
    ref.close_bf16(out.cpu()[own], want[own], noise[own])
    if lse is not None:
        got, w, e = lse.cpu().to(F64)[own], want_l[own], noise_l[own]
        none = torch.isinf(w)
        assert torch.equal(got[none], w[none])
        bad = ~((got[~none] - w[~none]).abs() <= e[~none])
        assert not bad.any(), float(((got - w).abs() / e)[~none].max())
