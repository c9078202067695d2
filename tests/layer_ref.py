"""The layer operators in 64 bits, from their definitions, for small sizes.

E4M3 decoding and rounding are written out here (no code shared with the
library), so are the dynamic scales.  `noise` arguments and results bound what
fp32 arithmetic may do to a value: U is the unit roundoff of fp32.  A kernel may
chain or tree its sums as it likes, so a sum of n terms is given n roundings of
the sum of the terms' magnitudes.
"""
from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24
BF16 = 2.0 ** -8  # half a step of bf16, relative to the value


def e4m3_values() -> torch.Tensor:
    """The 256 values of the E4M3FN bytes."""
    b = torch.arange(256)
    sign = torch.where(b >= 128, -1.0, 1.0).to(F64)
    e, m = (b >> 3) & 15, (b & 7).to(F64)
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).to(F64)))
    v = sign * v
    v[(b & 127) == 127] = float("nan")
    return v


_VALUES = e4m3_values()


def decode(bytes_: torch.Tensor) -> torch.Tensor:
    return _VALUES[bytes_.cpu().view(torch.uint8).long()]


def e4m3(v: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value, ties to even, saturating at 448."""
    a = v.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / step) * step, v).clamp(-448.0, 448.0)


def widen(s: torch.Tensor) -> torch.Tensor:
    return s.repeat_interleave(128, -1)


def scale(v: torch.Tensor) -> torch.Tensor:
    """fp32 scale of each 1x128 group: max(amax, 1e-4) / 448."""
    a = v.unflatten(-1, (-1, 128)).abs().amax(-1)
    floor = torch.tensor(1e-4, dtype=torch.float32).to(F64)
    return (torch.maximum(a, floor) / 448).float().to(F64)


def quantise_bf16(x: torch.Tensor):
    """(values, scales) of bf16 rows: exact amax, binary32 scale and quotient."""
    s = scale(x.to(F64))
    return e4m3((x.to(F64) / widen(s)).float().to(F64)), s


def tie_groups(n: int, g: torch.Generator) -> torch.Tensor:
    """n groups of 128 bf16 values (in fp32): the largest of each is an 8-bit whole
    number, and among the others are all whose E4M3 value of the binary32 quotient
    x / s differs from that of x times the binary32 reciprocal of s."""
    out = torch.empty((n, 128))
    for i in range(n):
        a = 128 + i % 128
        m = torch.arange(128, 256)[:, None] * torch.exp2(-torch.arange(9.0))
        v = m.flatten()[m.flatten() <= a]
        s = torch.tensor(float(a)) / torch.tensor(448.0)
        inv = (1 / s.to(F64)).float()
        moved = v[e4m3((v / s).to(F64)) != e4m3((v * inv).to(F64))][:100]
        rest = v[torch.randint(0, len(v), (127 - len(moved),), generator=g)]
        sign = torch.randint(0, 2, (127,), generator=g) * 2 - 1
        out[i, 0] = a
        out[i, 1:] = torch.cat([moved, rest]) * sign
    return out


def word_bytes(words: torch.Tensor) -> torch.Tensor:
    """The bytes of int32 rows, little-endian: [rows, 4 * columns]."""
    w = words.cpu().long()
    return torch.stack([(w >> b) & 255 for b in (0, 8, 16, 24)], -1).flatten(1)


def ue8m0(words: torch.Tensor, groups: int) -> torch.Tensor:
    """Scale values of row-major packed UE8M0 words [rows, P]."""
    return torch.exp2(word_bytes(words)[:, :groups].to(F64) - 127)


def mn_to_rows(words: torch.Tensor, rows: int, slab=None) -> torch.Tensor:
    """MN-major words ([P, stride], or [E, P, stride] with slab=(E, cap)) -> [rows, P]."""
    w = words.cpu()
    if slab is None:
        return w[:, :rows].T.contiguous()
    return w[:, :, :slab[1]].transpose(1, 2).reshape(rows, -1).contiguous()


def block_product(x, sx, w, sw):
    """(y, noise) of rows [m, K] (values, scales) with one expert's weights [N, K]."""
    a = x * widen(sx)
    b = w * widen(sw.to(F64).repeat_interleave(128, 0)[:w.shape[0]])
    # 128 products in a block, G blocks, the scales' product and its use
    n = 128 + sx.shape[-1] + 4
    return a @ b.T, 2 * n * U * (a.abs() @ b.abs().T)


def gated(y, noise):
    """(h, noise) of silu(gate) * up for y = [gate | up]."""
    g, u = y.chunk(2, -1)
    ng, nu = noise.chunk(2, -1)
    sig = 1 / (1 + torch.exp(-g))
    h = g * sig * u
    # |silu'| <= 1.1; exp of an fp32 number is off by a few roundings of g
    return h, 1.1 * ng * u.abs() + (g * sig).abs() * nu + h.abs() * (16 + 4 * g.abs()) * U + 1e-37


def spread(h, noise, power=False):
    """What the 8-bit rows of h (known to +-noise) may hold: (lo, hi, s_lo, s_hi)
    with q * s for each element between lo and hi.  power: UE8M0 scales."""
    a = h.unflatten(-1, (-1, 128)).abs()
    n = noise.unflatten(-1, (-1, 128))
    floor = torch.tensor(1e-4, dtype=torch.float32).to(F64)
    s_lo = torch.maximum((a - n).amax(-1), floor) / 448 * (1 - 4 * U)
    s_hi = torch.maximum((a + n).amax(-1), floor) / 448 * (1 + 4 * U)
    if power:
        s_lo, s_hi = (torch.exp2(torch.ceil(torch.log2(s))) for s in (s_lo, s_hi))
    c = []
    for s in (s_lo, s_hi):
        for v in (h - noise, h + noise):
            r = v / widen(s)
            for k in (1 - 2 * U, 1 + 2 * U):
                for m in (s_lo, s_hi):
                    c.append(e4m3(r * k) * widen(m))
    c = torch.stack(c)
    return c.amin(0), c.amax(0), s_lo, s_hi


def close_bf16(got, want, noise):
    """Assert |got - want| within bf16's half step plus the noise (itself rounded)."""
    got = got.to(F64).cpu()
    bound = want.abs() * BF16 + noise * (1 + BF16) + 2.0 ** -133
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / bound).max()))
