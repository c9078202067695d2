"""ep_expert_gemm and ep_expert_swiglu against the formula in 64 bits, on rows
that ep_layout and ep_dispatch made; tolerances are layer_ref's bounds of fp32
sums plus half a step of the output's type."""
import pytest
import torch

from combine_expert_histogram_gb300 import binding as ep
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

SENTINEL = 0x5A


def picks(T, E, K, seed, drop=0.1, only=None):
    g = torch.Generator().manual_seed(seed)
    pool = torch.arange(E) if only is None else torch.tensor(only)
    z = torch.rand((T, len(pool)), generator=g)
    idx = pool[z.argsort(1)[:, :min(K, len(pool))]]
    if idx.shape[1] < K:
        idx = torch.cat([idx, torch.full((T, K - idx.shape[1]), -1)], 1)
    idx = torch.where(torch.rand((T, K), generator=g) < drop, -1, idx)
    return idx.to(torch.int32)


def weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((E, N, K), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand((E, (N + 127) // 128, K // 128), generator=g) + 0.5) / (100 * K ** 0.5)
    return w.view(torch.uint8), s


class Case:
    """Rows of a dispatched batch, on the device and as (values, scales) in 64 bits."""

    def __init__(self, T, E, K, H, kind="contig", align=128, cap=0, quant="fp8_f32", seed=0,
                 drop=0.1, only=None):
        self.E, self.H, self.quant, self.kind, self.cap = E, H, quant, kind, cap
        idx = picks(T, E, K, seed, drop, only).cuda()
        g = torch.Generator().manual_seed(seed + 1)
        x = torch.randn((T, H), generator=g).bfloat16()
        L = self.L = ep.ep_layout(idx, E, kind=kind, align=align, capacity=cap)
        n = max(L.rows_capacity, 1)
        self.slab = (E, cap) if kind == "masked" else None
        self.x = torch.full((n, H), 0x7F, dtype=torch.uint8, device="cuda")  # NaN
        self.sx = ep.scale_buffer(L, H, quant)
        self.sx.fill_(float("nan")) if quant == "fp8_f32" else self.sx.fill_(-1)
        ep.ep_dispatch(L, x.cuda(), quant, out_rows=self.x, out_scales=self.sx)
        self.status = int(L.status.item())  # an overflowing slab says so
        self.n = n
        self.values = ref.decode(self.x)
        self.scales = self.scale_values(self.sx, H, quant)
        count, off = L.expert_count.tolist(), L.expert_offset.tolist()
        self.rows = [(off[e], min(count[e], cap) if kind == "masked" else count[e])
                     for e in range(E)]

    def scale_values(self, s, H, quant):
        if quant == "fp8_f32":
            return s.cpu().to(ref.F64)
        words = ref.mn_to_rows(s, self.n, self.slab) if quant == "fp8_ue8m0_mn" else s
        return ref.ue8m0(words, H // 128)

    def products(self, w, sw):
        """(first, rows, y, noise) of each expert that has rows."""
        for e, (a, n) in enumerate(self.rows):
            if n:
                y = ref.block_product(self.values[a:a + n], self.scales[a:a + n],
                                      ref.decode(w[e]), sw[e].cpu())
                yield a, n, *y

    def unused(self):
        free = torch.ones(self.n, dtype=torch.bool)
        for a, n in self.rows:
            free[a:a + n] = False
        return free


def check_gemm(c, N, seed=3):
    w, sw = weights(c.E, N, c.H, seed)
    out = torch.full((c.n, 2 * N), SENTINEL, dtype=torch.uint8, device="cuda").view(torch.bfloat16)
    keep = out.clone()
    got = ep.ep_expert_gemm(c.L, c.x, c.sx, w.cuda(), sw.cuda(), c.quant, out=out)
    torch.cuda.synchronize()
    assert int(c.L.status.item()) == c.status
    for a, n, y, noise in c.products(w, sw):
        ref.close_bf16(got[a:a + n], y, noise)
    free = c.unused()
    assert torch.equal(got.cpu().view(torch.int16)[free], keep.cpu().view(torch.int16)[free])


def check_swiglu(c, I, out_quant, seed=3):
    w, sw = weights(c.E, 2 * I, c.H, seed)
    plain = out_quant == "none"
    width = 2 * I if plain else I
    rows = torch.full((c.n, width), SENTINEL, dtype=torch.uint8, device="cuda")
    rows = rows.view(torch.bfloat16) if plain else rows
    scales = None
    if not plain:
        scales = ep.scale_buffer(c.L, I, out_quant)
        scales.view(torch.uint8).fill_(SENTINEL)
    keep, keep_s = rows.clone(), None if plain else scales.clone()
    got, got_s = ep.ep_expert_swiglu(c.L, c.x, c.sx, w.cuda(), sw.cuda(), c.quant, out_quant,
                                     out_rows=rows, out_scales=scales)
    torch.cuda.synchronize()
    assert int(c.L.status.item()) == c.status
    if not plain:
        values, s = ref.decode(got), c.scale_values(got_s, I, out_quant)
    for a, n, y, noise in c.products(w, sw):
        h, nh = ref.gated(y, noise)
        if plain:
            ref.close_bf16(got[a:a + n], h, nh)
            continue
        lo, hi, s_lo, s_hi = ref.spread(h, nh, power=out_quant != "fp8_f32")
        sg = s[a:a + n]
        assert ((sg >= s_lo * (1 - ref.U)) & (sg <= s_hi * (1 + ref.U))).all()
        v = values[a:a + n] * ref.widen(sg)
        slack = v.abs() * 4 * ref.U
        assert ((v >= lo - slack) & (v <= hi + slack)).all()
    free = c.unused()
    as_bytes = lambda t: t.cpu().view(torch.uint8)  # noqa: E731
    assert torch.equal(as_bytes(got)[free], as_bytes(keep)[free])
    if not plain and out_quant != "fp8_ue8m0_mn":
        assert torch.equal(as_bytes(got_s)[free], as_bytes(keep_s)[free])
    if not plain and out_quant.startswith("fp8_ue8m0"):
        words = ref.mn_to_rows(got_s, c.n, c.slab) if out_quant == "fp8_ue8m0_mn" else got_s
        b = ref.word_bytes(words)
        assert (b[~free][:, I // 128:] == 127).all()


LAYOUTS = [dict(kind="contig", align=128), dict(kind="contig", align=1),
           dict(kind="contig", align=16), dict(kind="masked", cap=32),
           dict(kind="masked", cap=5), dict(kind="masked", cap=131)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0", "fp8_ue8m0_mn"])
def test_gemm_layouts(layout, quant):
    check_gemm(Case(70, 6, 2, 640, quant=quant, seed=1, **layout), 264)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("out_quant", ["none", "fp8_f32", "fp8_ue8m0", "fp8_ue8m0_mn"])
def test_swiglu_layouts(layout, out_quant):
    check_swiglu(Case(70, 6, 2, 640, quant="fp8_f32", seed=2, **layout), 384, out_quant)


@pytest.mark.parametrize("quant", ["fp8_ue8m0", "fp8_ue8m0_mn"])
def test_swiglu_of_power_of_two_scales(quant):
    check_swiglu(Case(40, 5, 3, 1152, quant=quant, seed=3), 128, "fp8_f32")


@pytest.mark.parametrize("N", [8, 16, 120, 128, 136, 248, 256, 264, 520, 1000])
def test_gemm_widths(N):
    check_gemm(Case(33, 3, 2, 256, seed=N), N)


def test_widest_outputs():
    check_gemm(Case(5, 2, 1, 128, seed=19, drop=0.0), 65536)
    check_swiglu(Case(5, 2, 1, 128, seed=20, drop=0.0), 32768, "fp8_ue8m0")


@pytest.mark.parametrize("H", [128, 256, 384, 512, 896, 1408, 2048])
def test_gemm_inner_lengths(H):
    check_gemm(Case(20, 4, 2, H, seed=H), 136)
    check_swiglu(Case(20, 4, 2, H, seed=H + 1), 256, "fp8_f32")


@pytest.mark.parametrize("T", [1, 2, 127, 128, 129, 255, 257, 400])
def test_one_expert_with_every_row(T):
    """A one-expert layout: the product of a dense layer, any number of rows."""
    check_gemm(Case(T, 1, 1, 256, align=1, seed=T, drop=0.0), 136)


@pytest.mark.parametrize("T", [1, 130])
def test_one_expert_swiglu(T):
    check_swiglu(Case(T, 1, 1, 384, align=1, seed=T, drop=0.0), 128, "fp8_f32")


def test_many_experts_most_of_them_empty():
    check_gemm(Case(50, 1024, 2, 128, align=8, seed=5, only=[0, 3, 500, 1023]), 64)
    check_swiglu(Case(50, 1024, 2, 128, kind="masked", cap=20, seed=6, only=[1, 1022]), 128,
                 "fp8_f32")


def test_no_rows_at_all():
    check_gemm(Case(9, 4, 2, 128, seed=7, drop=2.0), 64)
    c = Case(0, 4, 2, 128, seed=8)
    check_gemm(c, 64)
    check_swiglu(c, 128, "fp8_f32")


@pytest.mark.parametrize("layout", [dict(kind="contig", align=128), dict(kind="contig", align=1)],
                         ids=str)
def test_more_tiles_than_processors(layout):
    """Several tiles for every SM, of experts with none to several row tiles."""
    c = Case(900, 40, 4, 256, seed=16, drop=0.05, only=list(range(0, 40, 2)) + [1], **layout)
    check_gemm(c, 1288)
    check_swiglu(c, 640, "fp8_f32")


@pytest.mark.parametrize("layout", [dict(kind="contig", align=128), dict(kind="contig", align=1),
                                    dict(kind="masked", cap=300)], ids=str)
@pytest.mark.parametrize("N", [136, 264, 520])
def test_several_row_tiles_an_expert(layout, N):
    """Odd and even numbers of row tiles and of weight tiles, an expert without
    rows, an overflowing slab."""
    c = Case(700, 4, 2, 384, seed=N, drop=0.05, only=[0, 1, 3], **layout)
    check_gemm(c, N)
    check_swiglu(c, {136: 128, 264: 256, 520: 384}[N], "fp8_f32")


@pytest.mark.parametrize("T", [256, 384, 513, 1000])
def test_several_row_tiles_of_one_expert(T):
    check_gemm(Case(T, 1, 1, 256, align=1, seed=T, drop=0.0, quant="fp8_ue8m0"), 1032)


@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0"])
def test_longest_rows(quant):
    c = Case(9, 2, 1, 32768, quant=quant, seed=17, drop=0.0)
    check_gemm(c, 264)


def test_captured_chain_replayed_on_new_inputs():
    """layout -> dispatch -> swiglu -> product -> combine in one graph."""
    T, E, K, H, I = 24, 6, 2, 384, 256
    dev = torch.device("cuda")
    idx = torch.zeros((T, K), dtype=torch.int32, device=dev)
    wt = torch.ones((T, K), device=dev)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=dev)
    w13, s13, w2, s2 = (t.cuda() for p in (weights(E, 2 * I, H, 1), weights(E, H, I, 2)) for t in p)
    L = ep.new_layout(T, K, E, "masked", capacity=T)
    n = L.rows_capacity
    rows = torch.empty((n, H), dtype=torch.uint8, device=dev)
    sc = ep.scale_buffer(L, H, "fp8_f32")
    h = torch.empty((n, I), dtype=torch.uint8, device=dev)
    sh = ep.scale_buffer(L, I, "fp8_f32")
    y = torch.empty((n, H), dtype=torch.bfloat16, device=dev)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    s = torch.cuda.Stream()

    def chain():
        ep.ep_layout(idx, E, out=L, stream=s)
        ep.ep_dispatch(L, x, "fp8_f32", out_rows=rows, out_scales=sc, stream=s)
        ep.ep_expert_swiglu(L, rows, sc, w13, s13, out_rows=h, out_scales=sh, stream=s)
        ep.ep_expert_gemm(L, h, sh, w2, s2, out=y, stream=s)
        ep.ep_combine(L, y, wt, out=out, stream=s)

    torch.cuda.synchronize()
    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        chain()
    for seed in (1, 2, 3):
        gen = torch.Generator().manual_seed(seed)
        idx.copy_(picks(T, E, K, seed))
        x.copy_(torch.randn((T, H), generator=gen).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        chain()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and not out.isnan().any()
        # the few-token layer computes the same without the chain's bf16 rounding
        # of each expert's output (half a step of each, added up)
        few = ep.ep_moe_decode(x, idx, wt, w13, s13, w2, s2).double()
        big = ep.ep_combine(L, y.abs(), wt).double()
        assert ((few - out.double()).abs() <= 2.1 * ref.BF16 * big + 2 * ref.BF16 * few.abs()).all()


@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0", "fp8_ue8m0_mn"])
def test_repacked_slab(quant):
    """A contiguous dispatch repacked into the slab: the product of the slab's rows
    is the product of the contiguous ones."""
    c = Case(60, 5, 2, 384, quant=quant, seed=18)
    cap = 40
    slab, ss, m = ep.ep_masked_repack(c.L, c.x, c.sx, quant, cap)
    M = ep.new_layout(60, 2, 5, "masked", capacity=cap)
    M.expert_count = m
    w, sw = (t.cuda() for t in weights(5, 136, 384, 3))
    a = ep.ep_expert_gemm(c.L, c.x, c.sx, w, sw, quant)
    b = ep.ep_expert_gemm(M, slab, ss, w, sw, quant).view(5, cap, 136)
    for e, (first, n) in enumerate(c.rows):
        assert n <= cap and torch.equal(a[first:first + n], b[e, :n])


def test_a_made_up_slab_of_a_batch_without_tokens():
    """Only the counts, the status and the slab's shape describe a made-up masked
    layout: its product is there although no token of this process is."""
    E, cap, K, N, I = 3, 20, 256, 136, 128
    c = Case(30, E, 2, K, kind="masked", cap=cap, seed=21)
    i32 = dict(dtype=torch.int32, device="cuda")
    made = ep.Layout(0, 0, E, 0, "masked", 0, cap, 0, dst_row=None, row_src=None,
                     expert_count=c.L.expert_count, expert_offset=None, rank_rows=None,
                     status=torch.zeros(1, **i32))
    empty = ep.new_layout(0, 2, E, "masked", capacity=cap)
    empty.expert_count = c.L.expert_count
    (w, sw), (wg, sg) = ([t.cuda() for t in weights(E, n, K, 3)] for n in (N, 2 * I))
    used = (~c.unused()).cuda()
    want = ep.ep_expert_gemm(c.L, c.x, c.sx, w, sw)[used]
    want_g = [t[used] for t in ep.ep_expert_swiglu(c.L, c.x, c.sx, wg, sg)]
    assert want.shape[0] > 20
    for L in (made, empty):
        assert torch.equal(ep.ep_expert_gemm(L, c.x, c.sx, w, sw)[used], want)
        got = ep.ep_expert_swiglu(L, c.x, c.sx, wg, sg)
        assert torch.equal(got[0][used], want_g[0]) and torch.equal(got[1][used], want_g[1])
        assert int(L.status.item()) == 0


def test_a_slab_of_no_tokens_writes_nothing():
    c = Case(0, 4, 2, 128, kind="masked", cap=6, seed=22)
    check_gemm(c, 64)
    check_swiglu(c, 128, "fp8_f32")


@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0", "fp8_ue8m0_mn"])
def test_gated_rows_are_quantised_by_the_rule_of_dispatch(quant):
    """Gates of 64 (silu(64) is 64 in fp32) and whole up sums of 8 bits: h is a
    bf16 number, so the 8-bit rows and scales are ep_dispatch's of the bf16 output,
    bit for bit.  The up values hold the quotients that ref.tie_groups picks."""
    groups, K, T = 128, 256, 5
    I = groups * 128
    g = torch.Generator().manual_seed(23)
    u = ref.tie_groups(groups, g).flatten()
    u[7 * 128:8 * 128] = 0.0
    # an 8-bit number is two E4M3 numbers of four bits
    unit = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=0.5))) - 3)
    hi = torch.trunc(u / unit) * unit
    w = torch.zeros((1, 2 * I, K))
    w[0, :I, 2] = 64.0
    w[0, I:, 0], w[0, I:, 1] = hi, u - hi
    f8 = w.to(torch.float8_e4m3fn)
    assert torch.equal(f8.float(), w)
    x = torch.zeros((T, K))
    x[:, 0], x[:, 2] = torch.tensor([1.0, -1, 1, 2, -0.5]), 1.0
    x[:, 1] = x[:, 0]
    L = ep.ep_layout(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1, align=1)
    one = torch.ones
    args = (L, x.to(torch.float8_e4m3fn).view(torch.uint8).cuda(), one(T, K // 128).cuda(),
            f8.view(torch.uint8).cuda(), one(1, 2 * I // 128, K // 128).cuda())
    out, _ = ep.ep_expert_swiglu(*args, out_quant="none")
    assert torch.equal(out.cpu().float(), 64 * x[:, :1] * u)
    rows, scales = ep.ep_expert_swiglu(*args, out_quant=quant)
    want, want_s, _ = ep.ep_dispatch(L, out, quant)
    # h of a zero up sum may have either sign
    as_bytes = lambda t: t.cpu().view(torch.uint8)  # noqa: E731
    zero = out.cpu() == 0
    assert torch.equal(as_bytes(rows)[~zero], as_bytes(want)[~zero])
    assert (as_bytes(rows)[zero] & 127 == 0).all()
    if quant == "fp8_ue8m0_mn":
        scales, want_s = scales[:, :T].contiguous(), want_s[:, :T].contiguous()
    assert torch.equal(as_bytes(scales), as_bytes(want_s))


def test_gate_within_its_stated_bound():
    """Exact gates from -448 to 448, close around where exp(-g) leaves fp32, and
    exact up sums from 2^-20 to 2^120: |h - formula| <= (16 + 4 |g|) 2^-24 |h| +
    2^-119 |u|, and half a step of bf16."""
    groups, K = 16, 128
    I = groups * 128
    gen = torch.Generator().manual_seed(24)
    v = ref.e4m3_values()
    v = v[~v.isnan()]
    near = -torch.tensor([80.0, 88, 88, 88, 96, 104]).to(ref.F64)
    a = torch.cat([near.repeat(64), v[torch.randint(0, len(v), (I - 384,), generator=gen)]])
    b = v[torch.randint(0, len(v), (I,), generator=gen)]
    b[:384] = torch.arange(384).remainder(65) / 16 - 2  # steps of 1/16 of four bits and a sign
    b = ref.e4m3(b)
    up = v[torch.randint(0, len(v), (I,), generator=gen)]
    up[::7] = 1.0
    w = torch.zeros((1, 2 * I, K))
    w[0, :I, 0], w[0, :I, 1], w[0, I:, 2] = a.float(), b.float(), up.float()
    power = torch.tensor([0, 100, 120, -20])[torch.arange(groups) % 4].to(ref.F64)
    scales = torch.cat([torch.ones(groups, dtype=ref.F64), torch.exp2(power)])
    x = torch.zeros((1, K))
    x[0, :3] = 1.0
    f8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    L = ep.ep_layout(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1, align=1)
    out, _ = ep.ep_expert_swiglu(L, f8(x), torch.ones((1, 1), device="cuda"), f8(w),
                                 scales.float().view(1, -1, 1).cuda(), out_quant="none")
    g, u = a + b, up * torch.exp2(power).repeat_interleave(128)
    h = g / (1 + torch.exp(-g)) * u
    noise = (16 + 4 * g.abs()) * ref.U * h.abs() + 2.0 ** -119 * u.abs()
    assert ((g < -86) & (g > -89) & (u.abs() > 2.0 ** 90)).sum() > 20
    # the bound is on fp32 numbers: 448 * 2^120 is none (2^128.8), nor are some of h;
    # there fp32 arithmetic gives an infinity, or NaN of one times zero
    fits = (u.abs() <= torch.finfo(torch.float32).max) & (h.abs() <= torch.finfo(torch.bfloat16).max)
    assert fits.sum() > 1800 and not out[0].cpu()[~fits].isfinite().any()
    ref.close_bf16(out[0].cpu()[fits], h[fits], noise[fits])


def test_first_call_of_a_process_is_captured():
    """Nothing of the first call (kernel attributes, the driver's encoder, lazy
    loading) is forbidden during a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    child = (
        "import sys; sys.path.insert(0, %r)\n"
        "import torch\n"
        "from combine_expert_histogram_gb300 import binding as ep\n"
        "d = dict(device='cuda')\n"
        "x = torch.randn(4, 256, **d).bfloat16(); n = torch.ones(256, **d).bfloat16()\n"
        "idx = torch.tensor([[0, 1]] * 4, dtype=torch.int32, **d); w = torch.ones(4, 2, **d)\n"
        "w13 = torch.full((2, 512, 256), 0x38, dtype=torch.uint8, **d)\n"
        "w2 = torch.full((2, 256, 256), 0x38, dtype=torch.uint8, **d)\n"
        "s13 = torch.full((2, 4, 2), 1e-2, **d); s2 = torch.full((2, 2, 2), 1e-2, **d)\n"
        "ws = ep.new_moe_workspace(4, 2, 2, 256, 256)\n"
        "out = torch.zeros_like(x); y = torch.zeros_like(x)\n"
        "torch.cuda.synchronize(); s = torch.cuda.Stream(); g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g, stream=s):\n"
        "    ep.ep_rmsnorm(x, n, out=y, stream=s)\n"
        "    ep.ep_moe_decode(y, idx, w, w13, s13, w2, s2, ws, out=out, stream=s)\n"
        "g.replay(); torch.cuda.synchronize(); got = out.clone()\n"
        "want = ep.ep_moe_decode(ep.ep_rmsnorm(x, n)[0], idx, w, w13, s13, w2, s2)\n"
        "torch.cuda.synchronize(); assert torch.equal(got, want) and got.abs().sum() > 0\n"
        "print('ok')\n" % root)
    r = subprocess.run([sys.executable, "-c", child], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_sums_keep_24_bits():
    """Integers whose block sums stay below 2^24 in any order: every partial sum
    is an fp32 number, so the result has no error but the final rounding."""
    E, H, N, T = 2, 256, 128, 40
    g = torch.Generator().manual_seed(9)
    L = ep.ep_layout(torch.arange(T, dtype=torch.int32).remainder(E)[:, None].cuda(), E, align=1)
    n = L.rows_capacity
    small = torch.tensor([-3.0, -2, -1, 1, 2, 3])
    x = small[torch.randint(0, 6, (n, H), generator=g)]
    w = small[torch.randint(0, 6, (E, N, H), generator=g)]
    # +-448 * 448 pairs that cancel: 2^17.6 next to single units
    at = torch.randperm(128, generator=g)[:8]
    for b in (0, 128):
        x[:, at + b] = 448.0
        w[:, :, at[:4] + b] = 448.0
        w[:, :, at[4:] + b] = -448.0
    f8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    one = torch.ones
    got = ep.ep_expert_gemm(L, f8(x), one(n, H // 128).cuda(), f8(w),
                            one(E, 1, H // 128).cuda())
    off = L.expert_offset.tolist()
    for e in range(E):
        want = x[off[e]:off[e + 1]].double() @ w[e].double().T
        assert want.abs().max() < 2 ** 24
        assert torch.equal(got[off[e]:off[e + 1]].cpu(), want.bfloat16())


def test_infinite_and_nan_rows_stay_in_their_rows():
    c = Case(40, 3, 2, 256, align=1, seed=10, drop=0.0)
    a, n = c.rows[1]
    c.x[a, 17] = 0x7F
    w, sw = weights(3, 136, 256, 3)
    got = ep.ep_expert_gemm(c.L, c.x, c.sx, w.cuda(), sw.cuda())
    assert got[a].isnan().all()
    c.rows[1] = (a + 1, n - 1)
    for f, m, y, noise in c.products(w, sw):
        ref.close_bf16(got[f:f + m], y, noise)


def test_a_layout_that_was_never_filled_reads_and_writes_inside_its_rows():
    """Counts and offsets that no ep_layout wrote are clamped into the row space."""
    c = Case(10, 4, 2, 128, seed=11)
    w, sw = weights(4, 64, 128, 3)
    guard = torch.full((c.n + 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.L.expert_count.fill_(2 ** 30)
    c.L.expert_offset.copy_(torch.tensor([-5, 2 ** 30, c.n - 3, 0, 0], dtype=torch.int32))
    ep.ep_expert_gemm(c.L, c.x, c.sx, w.cuda(), sw.cuda(), out=guard[:c.n])
    torch.cuda.synchronize()
    assert (guard[c.n:] == 7.0).all()


@pytest.mark.parametrize("first", [-5, 0, "end - 3", 2 ** 30])
def test_one_expert_that_claims_more_rows_than_there_are(first):
    """One count of 2^30 is cut off at the end of the row space; the other experts
    have none."""
    c = Case(10, 4, 2, 128, seed=11)
    w, sw = weights(4, 264, 128, 3)
    first = c.n - 3 if first == "end - 3" else first
    guard = torch.full((c.n + 64, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    c.L.expert_count.copy_(torch.tensor([0, 0, 2 ** 30, 0], dtype=torch.int32))
    c.L.expert_offset.copy_(torch.tensor([0, 0, first, 0, 0], dtype=torch.int32))
    ep.ep_expert_gemm(c.L, c.x, c.sx, w.cuda(), sw.cuda(), out=guard[:c.n])
    torch.cuda.synchronize()
    a = min(max(first, 0), c.n)
    assert (guard[c.n:] == 7.0).all() and (guard[:a] == 7.0).all()
    assert (guard[a:c.n] != 7.0).any(1).all()


def test_the_same_call_twice_and_on_another_stream():
    c = Case(90, 5, 2, 512, seed=12)
    w, sw = (t.cuda() for t in weights(5, 512, 512, 3))
    a = ep.ep_expert_swiglu(c.L, c.x, c.sx, w, sw)
    b = ep.ep_expert_swiglu(c.L, c.x, c.sx, w, sw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    d = ep.ep_expert_swiglu(c.L, c.x, c.sx, w, sw, stream=s)
    torch.cuda.synchronize()
    used = (~c.unused()).cuda()
    for r in (b, d):
        assert torch.equal(a[0][used], r[0][used]) and torch.equal(a[1][used], r[1][used])


def test_two_streams_at_once():
    """Two products that overlap on the GPU share nothing."""
    cs = [Case(300, 8, 2, 1024, seed=s) for s in (13, 14)]
    ws = [[t.cuda() for t in weights(8, 640, 1024, s)] for s in (1, 2)]
    one = [ep.ep_expert_gemm(c.L, c.x, c.sx, *w) for c, w in zip(cs, ws)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.zeros_like(o) for o in one]
    for _ in range(5):
        for c, w, s, o in zip(cs, ws, streams, outs):
            ep.ep_expert_gemm(c.L, c.x, c.sx, *w, out=o, stream=s)
    torch.cuda.synchronize()
    for c, a, b in zip(cs, one, outs):
        used = (~c.unused()).cuda()
        assert torch.equal(a[used], b[used])


def test_refusals():
    c = Case(10, 4, 2, 256, seed=15)
    w, sw = (t.cuda() for t in weights(4, 256, 256, 3))
    ok = (c.L, c.x, c.sx, w, sw)
    ep.ep_expert_gemm(*ok)
    bad = [(c.x[1:], c.sx, w, sw), (c.x, c.sx[1:], w, sw), (c.x, c.sx, w[1:], sw),
           (c.x, c.sx, w, sw[1:]), (c.x, c.sx.double(), w, sw), (c.x.float(), c.sx, w, sw),
           (c.x, c.sx, w.cpu(), sw), (c.x, None, w, sw), (c.x, c.sx, w.transpose(1, 2), sw)]
    for args in bad:
        with pytest.raises(ValueError):
            ep.ep_expert_gemm(c.L, *args)
    for quant in ("none", "mxfp8"):
        with pytest.raises(ep.EPError) as e:
            ep.ep_expert_gemm(*ok, quant=quant)
        assert e.value.code == ep.EP_ERR_UNSUPPORTED
    with pytest.raises(ep.EPError):  # a width that is no multiple of 8
        ep.ep_expert_gemm(c.L, c.x, c.sx, w[:, :132].contiguous(), sw)
    with pytest.raises(ep.EPError):  # half of the width is no multiple of 128
        ep.ep_expert_swiglu(c.L, c.x, c.sx, w[:, :128].contiguous(), sw[:, :1].contiguous())
    with pytest.raises(ep.EPError):
        ep.ep_expert_swiglu(*ok, out_quant="mxfp8")
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(*ok, out=torch.empty(3, 256, dtype=torch.bfloat16, device="cuda"))
