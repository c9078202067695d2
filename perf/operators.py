"""Timed cases of the layer operators around dispatch and combine.

Three families: the RMS norm in front of a mixture-of-experts layer (with the
residual's addition and 8-bit output), the experts' block-scaled E4M3 products
on a layout's rows (plain and with the gated SiLU), and a whole
mixture-of-experts layer for a few tokens.  ``run`` computes a case in plain
torch operations, or through the package where ``own`` is set.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # one token of a decode step: launch latency
        dict(name="norm_one_token", op="norm", T=1, H=7168, residual=True, quant="fp8_f32"),
        # a batch of prompts of a large model: the memory's rate
        dict(name="norm_prefill", op="norm", T=16384, H=7168, residual=True, quant="fp8_f32"),
        # the first layer (no residual yet), a width that is no multiple of 128, an odd batch
        dict(name="norm_odd", op="norm", T=1021, H=2056, residual=False, quant="none"),
        # the up projection of prompts: about 512 rows for each of 256 experts
        dict(name="swiglu_prefill", op="gemm", act=True, kind="contig", align=128, cap=0, T=16384,
             E=256, K=8, H=7168, N=2048, quant="fp8_f32", skew=0.0),
        # the down projection of a smaller prompt, power-of-two scales
        dict(name="down_prefill", op="gemm", act=False, kind="contig", align=128, cap=0, T=8192,
             E=256, K=8, H=2048, N=7168, quant="fp8_ue8m0", skew=0.0),
        # a decode batch in the masked slab: about 16 rows for each expert
        dict(name="swiglu_decode", op="gemm", act=True, kind="masked", align=1, cap=256, T=256,
             E=128, K=8, H=2048, N=768, quant="fp8_f32", skew=0.0),
        # popular experts overflow their slots, others stay empty; a ragged inner length
        dict(name="down_skewed_slab", op="gemm", act=False, kind="masked", align=1, cap=64, T=300,
             E=64, K=6, H=1408, N=4096, quant="fp8_f32", skew=1.2),
        # segments that start anywhere, an output width that ends inside a block
        dict(name="gemm_ragged", op="gemm", act=False, kind="contig", align=1, cap=0, T=777, E=40,
             K=3, H=1280, N=1000, quant="fp8_f32", skew=0.8),
        # one token of a small model: latency
        dict(name="moe_one_token", op="moe", T=1, E=128, K=8, H=2048, I=768, drop=0.0),
        # a few tokens of a large model: almost every pick is an expert of its own
        dict(name="moe_8_tokens", op="moe", T=8, E=256, K=8, H=7168, I=2048, drop=0.0),
        # the largest few-token batch of a large model
        dict(name="moe_64_tokens", op="moe", T=64, E=256, K=8, H=7168, I=2048, drop=0.0),
        # odd sizes, entries that are not routed
        dict(name="moe_odd", op="moe", T=13, E=20, K=3, H=1152, I=640, drop=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "gemm", "moe"])
    if op == "norm":
        quant = rng.choice(["none", "fp8_f32"])
        unit = 8 if quant == "none" else 128
        return dict(op=op, T=_log(rng, 1, 16384), H=unit * max(1, _log(rng, 128, 8192) // unit),
                    residual=rng.random() < 0.7, quant=quant)
    if op == "gemm":
        act = rng.random() < 0.5
        kind = rng.choice(["contig", "masked"])
        E, T = _log(rng, 1, 256), _log(rng, 1, 4096)
        H = 128 * _log(rng, 1, 56)
        N = 128 * _log(rng, 1, 16) if act else 8 * _log(rng, 8, 896)
        return dict(op=op, act=act, kind=kind, align=rng.choice([1, 8, 128]),
                    cap=_log(rng, 1, 256) if kind == "masked" else 0, T=T, E=E,
                    K=rng.randint(1, min(8, E)), H=H, N=N,
                    quant=rng.choice(["fp8_f32", "fp8_ue8m0"]), skew=rng.choice([0.0, 0.6, 1.2]))
    E = _log(rng, 1, 256)
    return dict(op=op, T=_log(rng, 1, 64), E=E, K=rng.randint(1, min(8, E)),
                H=128 * _log(rng, 1, 56), I=128 * _log(rng, 1, 16),
                drop=rng.choice([0.0, 0.0, 0.3]))


def _active(E, entries):
    """Experts that a uniform router names at least once, on average."""
    return E * (1.0 - (1.0 - 1.0 / E) ** entries) if E > 1 else 1.0


def work(case):
    c = case
    if c["op"] == "norm":
        TH = c["T"] * c["H"]
        b = 2 * TH + 2 * c["H"] + 2 * TH + (4 * TH if c["residual"] else 0)
        if c["quant"] != "none":
            b += TH + TH // 32
        return {"bytes": b, "flops": 5 * TH}
    if c["op"] == "gemm":
        H, W = c["H"], c["N"] * (2 if c["act"] else 1)
        rows = c["T"] * c["K"]
        if c["kind"] == "masked":
            rows = min(rows, c["E"] * c["cap"])
        b = _active(c["E"], c["T"] * c["K"]) * W * H * (1 + 4 / 128 / 128)
        b += rows * (H + H / 32) + rows * (c["N"] * (1 + 1 / 32) if c["act"] else 2 * c["N"])
        return {"bytes": b, "flops": 2 * rows * W * H}
    entries = c["T"] * c["K"] * (1 - c["drop"])
    b = _active(c["E"], entries) * 3 * c["H"] * c["I"] + 4 * c["T"] * c["H"]
    return {"bytes": b, "flops": 6 * entries * c["H"] * c["I"]}


# ------------------------------------------------------------------- inputs
def _weights(g, E, N, K):
    """E4M3 weights of rows near N(0, 1/K), with a scale for each 128x128 block."""
    w = torch.empty((E, N, K), dtype=F8, device="cuda")
    for e0 in range(0, E, 64):
        n = min(64, E - e0)
        w[e0:e0 + n] = torch.randn((n, N, K), generator=g, device="cuda",
                                   dtype=torch.bfloat16).mul_(112).clamp_(-448, 448).to(F8)
    s = torch.rand((E, -(-N // 128), K // 128), generator=g, device="cuda") + 0.5
    return w.view(torch.uint8), s / (112 * math.sqrt(K))


def _picks(g, T, E, K, skew):
    """Distinct experts of each token; expert popularity falls like 1/rank^skew."""
    z = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)))
    z -= skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return torch.topk(z, K, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(device="cuda")
    s = {"case": c}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s["x"] = torch.randn((T, H), generator=g, **dev).bfloat16()
        # a residual stream grows with depth and has a few large channels
        s["residual"] = None
        if c["residual"]:
            r = 4 * torch.randn((T, H), generator=g, **dev)
            r[:, ::97] *= 8
            s["residual"] = r.bfloat16()
            s["residual_out"] = torch.empty_like(s["residual"])
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, **dev)).bfloat16()
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16, **dev)
        if c["quant"] != "none":
            s["rows"] = torch.empty((T, H), dtype=torch.uint8, **dev)
            s["scales"] = torch.empty((T, H // 128), **dev)
        return s
    if c["op"] == "moe":
        T, E, K, H, I = c["T"], c["E"], c["K"], c["H"], c["I"]
        s["x"] = torch.randn((T, H), generator=g, **dev).bfloat16()
        s["idx"] = _picks(g, T, E, K, 0.0)
        s["idx"][torch.rand((T, K), generator=g, **dev) < c["drop"]] = -1
        w = torch.rand((T, K), generator=g, **dev) + 0.1
        s["w"] = w / w.sum(1, keepdim=True)
        s["w13"], s["w13_scales"] = _weights(g, E, 2 * I, H)
        s["w2"], s["w2_scales"] = _weights(g, E, H, I)
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16, **dev)
        s["most"] = int(torch.bincount(s["idx"].flatten().long() + 1, minlength=E + 1)[1:].max())
        return s
    T, E, K, H, N = c["T"], c["E"], c["K"], c["H"], c["N"]
    idx = _picks(g, T, E, K, c["skew"])
    count = torch.bincount(idx.flatten().long(), minlength=E)
    if c["kind"] == "masked":
        cap = E * c["cap"]
        offset = torch.arange(E + 1, **dev) * c["cap"]
        used = count.clamp(max=c["cap"])
    else:
        cap = T * K + min(E, T * K) * (c["align"] - 1)
        padded = (count + c["align"] - 1) // c["align"] * c["align"]
        offset = torch.cat([torch.zeros(1, dtype=torch.int64, **dev), padded.cumsum(0)])
        used = count
    s["cap"], s["most"] = cap, int(used.max())
    s["count"], s["offset"] = count.to(torch.int32), offset.to(torch.int32)
    at = torch.arange(s["most"], **dev)[None, :]
    # the row of each (expert, slot); `cap` where the expert has no such slot
    s["slot"] = torch.where(at < used[:, None], offset[:E, None] + at, cap)
    s["dst_row"] = torch.full((max(T * K, 1),), -1, dtype=torch.int32, **dev)
    s["status"] = torch.zeros(1, dtype=torch.int32, **dev)
    # rows as dispatch leaves them: E4M3 up to 448 with one scale per 128, and
    # whatever was in memory (NaN here) in the rows that no entry fills
    x = torch.randn((cap, H), generator=g, dtype=torch.bfloat16, **dev).mul_(130).clamp_(-448, 448)
    x = x.to(F8).view(torch.uint8)
    sc = (torch.rand((cap, H // 128), generator=g, **dev) + 0.5) / 130
    if c["quant"] == "fp8_ue8m0":
        e = torch.floor(torch.log2(sc)).to(torch.int32) + 127
        e = torch.nn.functional.pad(e, (0, -(H // 128) % 4), value=127).view(cap, -1, 4)
        sc = (e * torch.tensor([1, 1 << 8, 1 << 16, 1 << 24], dtype=torch.int32, **dev)).sum(
            2).to(torch.int32)
    empty = torch.ones(cap + 1, dtype=torch.bool, **dev)
    empty[s["slot"].flatten()] = False
    x[empty[:cap]] = 0x7F
    sc[empty[:cap]] = float("nan") if sc.is_floating_point() else -1
    s["x"], s["x_scales"] = x, sc
    s["wt"], s["wt_scales"] = _weights(g, E, N * (2 if c["act"] else 1), H)
    if c["act"]:
        s["rows"] = torch.zeros((cap, N), dtype=torch.uint8, **dev)
        s["scales"] = torch.zeros((cap, N // 128), **dev)
    else:
        s["out"] = torch.zeros((cap, N), dtype=torch.bfloat16, **dev)
    return s


# --------------------------------------------------------------- plain form
def _quantise(v):
    """E4M3 values and fp32 scales of 1x128 groups, by IEEE divisions (torch
    multiplies by the reciprocal where the divisor is a plain number)."""
    g = v.unflatten(-1, (-1, 128))
    amax = g.abs().amax(-1).clamp_min(1e-4)
    sc = amax / torch.full_like(amax, 448.0)
    return (g / sc[..., None]).to(F8).flatten(-2), sc


def _dequantise(q, sc):
    return (q.float().unflatten(-1, (-1, 128)) * sc[..., None]).flatten(-2)


def _weight_values(w, sc):
    n = w.shape[-2]
    per_row = sc.repeat_interleave(128, dim=-2)[..., :n, :]
    return (w.view(F8).float().unflatten(-1, (-1, 128)) * per_row[..., None]).flatten(-2)


def _scale_values(s, groups):
    if s.is_floating_point():
        return s
    e = torch.stack([(s >> b) & 255 for b in (0, 8, 16, 24)], -1).flatten(-2)[:, :groups]
    return torch.exp2((e - 127).float())


def _gated(a):
    g, u = a.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _plain_norm(s):
    v = s["x"].float()
    r = {}
    if s["residual"] is not None:
        v = v + s["residual"].float()
        r["residual"] = v.bfloat16()
    y = v * (1.0 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)) * s["weight"].float()
    r["out"] = y.bfloat16()
    if s["case"]["quant"] != "none":
        r["rows"], r["scales"] = _quantise(y)
    return r


def _plain_gemm(s):
    c = s["case"]
    x = _dequantise(s["x"].view(F8), _scale_values(s["x_scales"], c["H"] // 128))
    x = torch.cat([x, x.new_zeros(1, c["H"])])
    a = torch.bmm(x[s["slot"]], _weight_values(s["wt"], s["wt_scales"]).transpose(1, 2))
    at = s["slot"].flatten()
    if c["act"]:
        q, sc = _quantise(_gated(a))
        rows = torch.zeros((s["cap"] + 1, c["N"]), dtype=torch.uint8, device=q.device)
        rows[at] = q.view(torch.uint8).flatten(0, 1)
        scales = sc.new_zeros((s["cap"] + 1, c["N"] // 128))
        scales[at] = sc.flatten(0, 1)
        rows, scales = rows[:s["cap"]], scales[:s["cap"]]
        return {"rows": rows.view(F8), "scales": scales}
    out = torch.zeros((s["cap"] + 1, c["N"]), dtype=torch.bfloat16, device=a.device)
    out[at] = a.bfloat16().flatten(0, 1)
    return {"out": out[:s["cap"]]}


def _plain_moe(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    x = _dequantise(*_quantise(s["x"].float()))
    idx = s["idx"].flatten().long()
    if T * K <= E // 2:  # the picked experts' weights, once for each entry
        e = idx.clamp_min(0)
        a = x.repeat_interleave(K, 0)[:, None]
        a = torch.bmm(a, _weight_values(s["w13"][e], s["w13_scales"][e]).transpose(1, 2))
        h = _dequantise(*_quantise(_gated(a)))
        y = torch.bmm(h, _weight_values(s["w2"][e], s["w2_scales"][e]).transpose(1, 2))[:, 0]
    else:  # all experts, each with up to `most` entries
        order = torch.argsort(idx, stable=True)
        first = torch.searchsorted(idx[order], torch.arange(E, device=idx.device))
        slot = torch.empty_like(idx)
        slot[order] = torch.arange(T * K, device=idx.device) - first[idx[order].clamp_min(0)]
        routed = idx >= 0
        at = torch.where(routed, idx * s["most"] + slot, E * s["most"])
        a = x.new_zeros((E * s["most"] + 1, c["H"]))
        a[at] = x.repeat_interleave(K, 0)
        a = a[:-1].view(E, s["most"], c["H"])
        a = torch.bmm(a, _weight_values(s["w13"], s["w13_scales"]).transpose(1, 2))
        h = _dequantise(*_quantise(_gated(a)))
        y = torch.bmm(h, _weight_values(s["w2"], s["w2_scales"]).transpose(1, 2)).flatten(0, 1)
        y = y[torch.where(routed, at, 0)]
    y = torch.where((idx >= 0)[:, None], y, 0.0).view(T, K, c["H"])
    return {"out": (y * s["w"][..., None]).sum(1).bfloat16()}


# ---------------------------------------------------------- the framework's
def _own_norm(s):
    from combine_expert_histogram_gb300 import binding as ep

    quant = s["case"]["quant"]
    out, rows, scales, res = ep.ep_rmsnorm(
        s["x"], s["weight"], EPS, residual=s["residual"], quant=quant, out=s["out"],
        out_rows=s.get("rows"), out_scales=s.get("scales"), residual_out=s.get("residual_out"))
    r = {"out": out}
    if res is not None:
        r["residual"] = res
    if rows is not None:
        r["rows"], r["scales"] = rows.view(F8), scales
    return r


def _own_gemm(s):
    from combine_expert_histogram_gb300 import binding as ep

    c = s["case"]
    if "layout" not in s:  # the handle that ep_layout would have filled
        s["layout"] = ep.Layout(
            c["T"], c["K"], c["E"], 1, c["kind"], c["align"], c["cap"], 0, dst_row=s["dst_row"],
            row_src=None, expert_count=s["count"], expert_offset=s["offset"], rank_rows=None,
            status=s["status"])
    if c["act"]:
        rows, scales = ep.ep_expert_swiglu(s["layout"], s["x"], s["x_scales"], s["wt"],
                                           s["wt_scales"], c["quant"], out_quant="fp8_f32",
                                           out_rows=s["rows"], out_scales=s["scales"])
        return {"rows": rows.view(F8), "scales": scales}
    return {"out": ep.ep_expert_gemm(s["layout"], s["x"], s["x_scales"], s["wt"], s["wt_scales"],
                                     c["quant"], out=s["out"])}


def _own_moe(s):
    from combine_expert_histogram_gb300 import binding as ep

    c = s["case"]
    if "ws" not in s:
        s["ws"] = ep.new_moe_workspace(c["T"], c["K"], c["E"], c["H"], c["I"])
    return {"out": ep.ep_moe_decode(s["x"], s["idx"], s["w"], s["w13"], s["w13_scales"], s["w2"],
                                    s["w2_scales"], s["ws"], out=s["out"])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "gemm": _own_gemm, "moe": _own_moe}[op](state)
    return {"norm": _plain_norm, "gemm": _plain_gemm, "moe": _plain_moe}[op](state)


# -------------------------------------------------------------- the 64 bits
def _e4m3(v):
    """Nearest E4M3 value (ties to even, saturating) of float64 values."""
    a = v.abs().clamp_max(448.0)
    e = torch.frexp(a).exponent.sub(1).clamp_min(-6)
    step = torch.exp2((e - 3).double())
    return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), v)


def _groups64(v):
    """(E4M3 values, scales) of the 1x128 groups of float64 rows.  The scale and
    the quotient are binary32 by the format's definition: bf16 inputs often lie
    within 2^-24 of a tie between two E4M3 values, which side is decided there."""
    sc = v.reshape(v.shape[0], -1, 128).abs().amax(2).clamp_min(1e-4) / 448
    sc = sc.float().double()
    wide = sc.repeat_interleave(128, 1)
    return _e4m3((v / wide).float().double()), sc


def _w64(w, sc):
    n, k = w.shape
    wide = sc.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return w.view(F8).double() * wide


def exact(case, seed):
    c = case
    w = work(c)
    if w["flops"] > 3e12 or w["bytes"] > 3e10:
        return None
    s = prepare(c, seed)
    if c["op"] == "norm":
        v = s["x"].double()
        r = {}
        if s["residual"] is not None:
            v += s["residual"].double()
            r["residual"] = v
        y = v / (v.pow(2).sum(1, keepdim=True) / c["H"] + EPS).sqrt() * s["weight"].double()
        r["out"] = y
        if c["quant"] != "none":
            r["rows"], r["scales"] = _groups64(y)
        return r
    if c["op"] == "moe":
        q, sc = _groups64(s["x"].double())
        x = q * sc.repeat_interleave(128, 1)
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for e in s["idx"].unique().tolist():
            if e < 0:
                continue
            t, k = torch.nonzero(s["idx"] == e, as_tuple=True)
            a = x[t] @ _w64(s["w13"][e], s["w13_scales"][e]).T
            gate, up = a[:, :c["I"]], a[:, c["I"]:]
            q, sc = _groups64(gate * torch.sigmoid(gate) * up)
            y = (q * sc.repeat_interleave(128, 1)) @ _w64(s["w2"][e], s["w2_scales"][e]).T
            out.index_add_(0, t, y * s["w"][t, k].double()[:, None])
        return {"out": out}
    groups = c["H"] // 128
    W = torch.float64
    if c["act"]:
        r = {"rows": torch.zeros((s["cap"], c["N"]), dtype=W, device="cuda"),
             "scales": torch.zeros((s["cap"], c["N"] // 128), dtype=W, device="cuda")}
    else:
        r = {"out": torch.zeros((s["cap"], c["N"]), dtype=W, device="cuda")}
    offset, count = s["offset"].tolist(), s["count"].tolist()
    for e in range(c["E"]):
        n = min(count[e], c["cap"]) if c["kind"] == "masked" else count[e]
        a, b = offset[e], offset[e] + n
        if n == 0:
            continue
        sc = s["x_scales"][a:b]
        if not sc.is_floating_point():
            byte = sc.contiguous().view(torch.uint8)[:, :groups]
            sc = torch.ldexp(torch.ones((), dtype=W, device="cuda"), byte.int() - 127)
        x = s["x"][a:b].view(F8).double() * sc.double().repeat_interleave(128, 1)
        y = x @ _w64(s["wt"][e], s["wt_scales"][e]).T
        if c["act"]:
            gate, up = y[:, :c["N"]], y[:, c["N"]:]
            r["rows"][a:b], r["scales"][a:b] = _groups64(gate * torch.sigmoid(gate) * up)
        else:
            r["out"][a:b] = y
    return r
