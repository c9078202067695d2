"""ep_moe_decode against the formula in 64 bits, and against the chain of
layout, dispatch, expert products and combine."""
import pytest
import torch

from combine_expert_histogram_gb300 import binding as ep
from tests import layer_ref as ref
from tests.test_gpu_expert import picks, weights

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


class Case:
    def __init__(self, T, E, K, H, I, seed=0, drop=0.1, idx=None, x=None):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn((T, H), generator=g).bfloat16() if x is None else x
        self.idx = picks(T, E, K, seed, drop) if idx is None else idx
        w = torch.rand((T, K), generator=g) + 0.05
        self.w = w / w.sum(1, keepdim=True)
        self.w13, self.s13 = weights(E, 2 * I, H, seed + 1)
        self.w2, self.s2 = weights(E, H, I, seed + 2)
        self.E = E
        self.dev = [t.cuda() for t in (self.x, self.idx, self.w, self.w13, self.s13, self.w2,
                                       self.s2)]

    def formula(self, q=None, s=None):
        """(out, noise): the noise includes 8-bit values that may fall on either
        side of a tie, and the workspace's and the combination's fp32 sums."""
        if q is None:
            q, s = ref.quantise_bf16(self.x)
        T, H = q.shape
        out = torch.zeros((T, H), dtype=ref.F64)
        noise = torch.zeros_like(out)
        K = self.idx.shape[1]
        for e in self.idx.unique().tolist():
            if not 0 <= e < self.E:
                continue
            t, k = torch.nonzero(self.idx == e, as_tuple=True)
            h, nh = ref.gated(*ref.block_product(q[t], s[t], ref.decode(self.w13[e]), self.s13[e]))
            lo, hi, s_lo, s_hi = ref.spread(h, nh)
            w2 = ref.decode(self.w2[e])
            mid, half = (lo + hi) / 2, (hi - lo) / 2
            one = torch.ones((len(t), mid.shape[1] // 128), dtype=ref.F64)
            y, ny = ref.block_product(mid, one, w2, self.s2[e])
            b = w2 * ref.widen(self.s2[e].to(ref.F64).repeat_interleave(128, 0))
            ny = ny + half @ b.abs().T
            wt = self.w[t, k].to(ref.F64)[:, None]
            out.index_add_(0, t, y * wt)
            noise.index_add_(0, t, wt * (ny + (K + 4) * ref.U * y.abs()))
        return out, noise * 1.01

    def check(self, out, **kw):
        ref.close_bf16(out, *self.formula(**kw))


@pytest.mark.parametrize("T,E,K,H,I", [
    (1, 8, 2, 128, 128), (1, 16, 8, 2048, 768), (1, 1, 1, 256, 128), (2, 4, 1, 384, 256),
    (3, 20, 5, 1152, 640), (8, 32, 8, 512, 256), (13, 20, 3, 640, 384), (16, 4, 2, 256, 512),
    (33, 6, 3, 384, 256), (64, 5, 4, 256, 128), (64, 1, 1, 256, 256), (100, 3, 2, 128, 384),
    (32, 1024, 32, 128, 128), (5, 8, 3, 1024, 2048), (1, 4, 2, 4096, 128), (4, 3, 2, 128, 4096)])
def test_formula(T, E, K, H, I):
    c = Case(T, E, K, H, I, seed=T + H)
    ws = ep.new_moe_workspace(T, K, E, H, I)
    c.check(ep.ep_moe_decode(*c.dev, ws))
    ws.check_status()


@pytest.mark.parametrize("dim", [dict(H=16384, I=128), dict(H=128, I=16384)], ids=str)
def test_largest_dimensions(dim):
    c = Case(3, 2, 2, seed=5, drop=0.0, **dim)
    c.check(ep.ep_moe_decode(*c.dev))


def test_every_token_to_one_expert():
    """More entries of one expert than any tile holds."""
    idx = torch.zeros((128, 8), dtype=torch.int32)
    c = Case(128, 4, 8, 128, 128, seed=3, idx=idx)
    c.check(ep.ep_moe_decode(*c.dev))


def test_repeated_unrouted_and_bad_ids():
    idx = torch.tensor([[1, 1, 1], [-1, -1, -1], [0, -1, 2], [7, 0, -5], [2, 2, 0]],
                       dtype=torch.int32)
    c = Case(5, 3, 3, 256, 256, seed=4, idx=idx)
    ws = ep.new_moe_workspace(5, 3, 3, 256, 256)
    out = ep.ep_moe_decode(*c.dev, ws)
    c.check(out)
    assert (out[1] == 0).all()
    with pytest.raises(ep.EPError) as e:
        ws.check_status()
    assert e.value.code == ep.EP_ERR_BAD_EXPERT_ID
    c.dev[1].clamp_(-1, 2)  # the next call starts from a clean status
    ep.ep_moe_decode(*c.dev, ws)
    ws.check_status()


def test_nothing_routed():
    idx = torch.full((4, 2), -1, dtype=torch.int32)
    c = Case(4, 3, 2, 128, 128, seed=4, idx=idx)
    out = torch.full((4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ep.ep_moe_decode(*c.dev, out=out)
    assert (out == 0).all() and not torch.signbit(out).any()


def test_nan_and_infinite_tokens_stay_with_their_token():
    g = torch.Generator().manual_seed(6)
    x = torch.randn((6, 256), generator=g).bfloat16()
    x[2, 9] = float("nan")
    x[4, 200] = float("inf")
    idx = torch.tensor([[0, 1]] * 6, dtype=torch.int32)
    c = Case(6, 2, 2, 256, 256, seed=6, idx=idx, x=x)
    out = ep.ep_moe_decode(*c.dev)
    keep = [0, 1, 3, 5]
    c.x[2], c.x[4] = 0, 0
    want, noise = c.formula()
    ref.close_bf16(out[keep], want[keep], noise[keep])
    assert out[2].isnan().any()


@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0"])
def test_8_bit_rows_of_the_norm(quant):
    """norm -> decode layer: the rows in 8 bits, as ep_rmsnorm writes them."""
    c = Case(7, 6, 3, 640, 256, seed=7)
    w = torch.ones(640, dtype=torch.bfloat16, device="cuda")
    _, q, s, _ = ep.ep_rmsnorm(c.dev[0], w, quant=quant, with_out=False)
    out = ep.ep_moe_decode(q, *c.dev[1:], x_scales=s, quant=quant)
    sv = s.cpu().to(ref.F64) if quant == "fp8_f32" else ref.ue8m0(s, 5)
    c.check(out, q=ref.decode(q), s=sv)


def test_workspace_left_dirty_and_shared_by_calls_in_a_row():
    a, b = Case(9, 6, 3, 256, 384, seed=8), Case(4, 6, 2, 256, 384, seed=9)
    ws = ep.new_moe_workspace(9, 3, 6, 256, 384)
    ws.scratch.fill_(0xFF)
    for _ in range(3):
        oa, ob = ep.ep_moe_decode(*a.dev, ws), ep.ep_moe_decode(*b.dev, ws)
    a.check(oa)
    b.check(ob)


def test_one_workspace_for_any_smaller_batch():
    """Batches from 1 to 40 tokens, on both sides of where rows are cut into parts."""
    c = Case(40, 64, 8, 256, 640, seed=21)
    x, idx, w = c.dev[:3]
    ws = ep.new_moe_workspace(40, 8, 64, 256, 640)
    want, noise = c.formula()
    for T in (1, 2, 3, 5, 8, 13, 21, 30, 39, 40):
        out = ep.ep_moe_decode(x[:T], idx[:T], w[:T], *c.dev[3:], ws)
        ref.close_bf16(out, want[:T], noise[:T])


def test_norm_straight_into_the_layer_and_on():
    """norm -> layer -> norm without a wait between them, many times over one set
    of buffers: every kernel waits for what it reads and for what it overwrites."""
    c = Case(3, 16, 4, 640, 384, seed=22, drop=0.0)
    res = c.dev[0].clone()
    wn = torch.ones(640, dtype=torch.bfloat16, device="cuda")
    ws = ep.new_moe_workspace(3, 4, 16, 640, 384)

    def step(sync):
        x, h, out = res.clone(), torch.empty_like(res), torch.zeros_like(res)
        seen = []
        for _ in range(6):
            ep.ep_rmsnorm(out, wn, residual=x, out=h, residual_out=x)
            if sync:
                torch.cuda.synchronize()
            ep.ep_moe_decode(h, *c.dev[1:], ws, out=out)
            if sync:
                torch.cuda.synchronize()
            seen.append(out.clone())
        return seen

    want = step(True)
    for _ in range(5):
        for a, b in zip(want, step(False)):
            assert torch.equal(a, b)


def test_the_same_bits_every_time():
    c = Case(24, 12, 4, 512, 384, seed=10)
    first = ep.ep_moe_decode(*c.dev)
    for _ in range(20):
        assert torch.equal(first, ep.ep_moe_decode(*c.dev))


def test_sums_keep_24_bits():
    """Integers next to cancelling pairs of 448 * 448: any fp32 order of the sums
    is exact, so the up product, its 8-bit form (values and scales chosen to be
    representable) and the down product have no error but the last rounding."""
    T, H, I = 8, 256, 128
    g = torch.Generator().manual_seed(20)
    x = torch.zeros((T, H))
    up, gate = torch.zeros((I, H)), torch.zeros((I, H))
    for b in (0, 128):
        at = torch.randperm(126, generator=g)[:8] + 2 + b
        x[:, at] = 448.0
        up[:, at[:4]], up[:, at[4:]] = 448.0, -448.0
    x[:, 0] = 1.0
    gate[:, 0] = 64.0  # silu(64) = 64 in fp32
    x[:, 1] = 1.0
    v = torch.cat([torch.arange(-15, 16), torch.arange(16, 32, 2)]).float()
    up[:, 1] = v[torch.randint(0, len(v), (I,), generator=g)]
    up[5, 1] = 448.0  # makes the scale of the gated group 64
    w2 = torch.randint(-4, 5, (H, I), generator=g).float()
    f8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)[None].cuda()  # noqa: E731
    one = torch.ones
    out = ep.ep_moe_decode(x.bfloat16().cuda(), torch.zeros((T, 1), dtype=torch.int32).cuda(),
                           one(T, 1).cuda(), f8(torch.cat([gate, up])), one(1, 2, 2).cuda(),
                           f8(w2), one(1, 2, 1).cuda())
    want = 64 * (up[:, 1].double() @ w2.double().T)
    assert torch.equal(out.cpu(), want.bfloat16().expand(T, H))


def test_two_streams_with_a_workspace_each():
    cs = [Case(8, 16, 4, 1024, 512, seed=s) for s in (11, 12)]
    one = [ep.ep_moe_decode(*c.dev) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [ep.new_moe_workspace(8, 4, 16, 1024, 512) for _ in cs]
    outs = [torch.zeros_like(o) for o in one]
    for _ in range(10):
        for c, s, w, o in zip(cs, streams, ws, outs):
            ep.ep_moe_decode(*c.dev, w, out=o, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(one, outs):
        assert torch.equal(a, b)


def test_all_operators_at_once_on_four_streams():
    """Blocks of the few-token layer (half an SM's shared memory, half its tensor
    memory), of the experts' products (all of both) and of the norm wait for one
    another's resources, never for each other."""
    from tests.test_gpu_expert import Case as Rows
    small, other = Case(5, 12, 4, 512, 384, seed=23), Case(40, 6, 4, 512, 384, seed=24)
    r = Rows(300, 8, 2, 768, seed=25)
    w, sw = (t.cuda() for t in weights(8, 512, 768, 26))
    x = torch.randn((700, 1024), device="cuda").bfloat16()
    g = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    ws = [ep.new_moe_workspace(5, 4, 12, 512, 384), ep.new_moe_workspace(40, 4, 6, 512, 384)]
    used = (~r.unused()).cuda()
    calls = [lambda s: ep.ep_moe_decode(*small.dev, ws[0], stream=s),
             lambda s: ep.ep_moe_decode(*other.dev, ws[1], stream=s),
             lambda s: ep.ep_expert_swiglu(r.L, r.x, r.sx, w, sw, out_quant="none", stream=s)[0][used],
             lambda s: ep.ep_rmsnorm(x, g, quant="fp8_f32", with_out=False, stream=s)[1]]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(c(s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    for q in ws:
        q.check_status()


def test_captured_and_replayed_on_new_inputs():
    c = Case(5, 8, 3, 384, 256, seed=13)
    ws = ep.new_moe_workspace(5, 3, 8, 384, 256)
    out = torch.empty((5, 384), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ep.ep_moe_decode(*c.dev, ws, out=out, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.ep_moe_decode(*c.dev, ws, out=out, stream=s)
    for seed in (14, 15):
        n = Case(5, 8, 3, 384, 256, seed=seed)
        for a, b in zip(c.dev, n.dev):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        n.check(out)


@pytest.mark.parametrize("T,kind", [(6, "contig"), (150, "contig"), (40, "masked")])
def test_a_layer_from_norm_to_combine(T, kind):
    """norm -> router -> layout -> dispatch -> swiglu -> product -> combine, as a
    prompt runs it, against the formula on the norm's own rows; for few tokens
    ep_moe_decode on the same rows gives the same layer."""
    E, K, H, I = 12, 3, 384, 256
    c = Case(T, E, K, H, I, seed=T)
    g = torch.Generator().manual_seed(T)
    res = torch.randn((T, H), generator=g).bfloat16().cuda()
    gate = (torch.randn((H, E), generator=g) / H ** 0.5).cuda()
    wn = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
    x, _, _, _ = ep.ep_rmsnorm(c.dev[0], wn, residual=res)
    idx, w = ep.ep_route_topk(x.float() @ gate, K)
    L = ep.ep_layout(idx, E, kind=kind, capacity=T)
    rows, sx, _ = ep.ep_dispatch(L, x, "fp8_f32")
    h, sh = ep.ep_expert_swiglu(L, rows, sx, *c.dev[3:5])
    y = ep.ep_expert_gemm(L, h, sh, *c.dev[5:7])
    out = ep.ep_combine(L, y, w)
    L.check_status()
    c.x, c.idx, c.w = x.cpu(), idx.cpu(), w.cpu()
    want, noise = c.formula()
    # the chain also rounds each expert's output to bf16 before the combination
    extra = torch.zeros_like(want)
    dst = L.dst_row.cpu().long()[:T * K].view(T, K)
    for k in range(K):
        extra += y.cpu()[dst[:, k]].to(ref.F64).abs() * c.w[:, k:k + 1].to(ref.F64) * ref.BF16
    ref.close_bf16(out, want, noise + 1.01 * extra)
    if T * K <= 1024:
        ref.close_bf16(ep.ep_moe_decode(x, idx, w, *c.dev[3:]), want, noise)


@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0", "fp8_ue8m0_mn"])
@pytest.mark.parametrize("T", [1, 6, 131])
def test_a_shared_expert_on_the_norms_rows(T, quant):
    """norm -> swiglu -> product of a one-expert layout: the norm's 8-bit rows as they
    are (token t is row t), in every scale format, with gated rows of the same; for
    the formats ep_moe_decode takes, it gives the same layer."""
    H, I = 640, 384
    c = Case(T, 1, 1, H, I, seed=T, idx=torch.zeros((T, 1), dtype=torch.int32))
    wn = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    _, q, s, _ = ep.ep_rmsnorm(c.dev[0], wn, quant=quant, with_out=False)
    L = ep.ep_layout(c.dev[1], 1, align=1)
    assert L.rows_capacity == T
    w13, s13, w2, s2 = c.dev[3:]
    h, sh = ep.ep_expert_swiglu(L, q, s, w13, s13, quant, out_quant="fp8_f32")
    y = ep.ep_expert_gemm(L, h, sh, w2, s2)
    c.w = torch.ones((T, 1))
    words = ref.mn_to_rows(s, T) if quant == "fp8_ue8m0_mn" else s
    sv = s.cpu().to(ref.F64) if quant == "fp8_f32" else ref.ue8m0(words, H // 128)
    c.check(y, q=ref.decode(q), s=sv)
    if quant != "fp8_ue8m0_mn":
        few = ep.ep_moe_decode(q, c.dev[1], torch.ones((T, 1), device="cuda"), *c.dev[3:],
                               x_scales=s, quant=quant)
        c.check(few, q=ref.decode(q), s=sv)


def test_refusals():
    c = Case(4, 4, 2, 256, 256, seed=16)
    x, idx, w, w13, s13, w2, s2 = c.dev
    ws = ep.new_moe_workspace(4, 2, 4, 256, 256)
    bad = [(x.float(), idx, w, w13, s13, w2, s2), (x, idx.long(), w, w13, s13, w2, s2),
           (x, idx, w.double(), w13, s13, w2, s2), (x, idx[1:], w, w13, s13, w2, s2),
           (x, idx, w, w13[1:], s13, w2, s2), (x, idx, w, w13, s13[1:], w2, s2),
           (x, idx, w, w13, s13, w2.transpose(1, 2), s2), (x, idx, w, w13, s13, w2, s2.cpu()),
           (x.t(), idx, w, w13, s13, w2, s2)]
    for args in bad:
        with pytest.raises(ValueError):
            ep.ep_moe_decode(*args, ws)
    with pytest.raises(ValueError):  # 8-bit rows without scales
        ep.ep_moe_decode(x.view(torch.uint8)[:, :256].contiguous(), *c.dev[1:], ws,
                         quant="fp8_f32")
    small = ep.MoeWorkspace(ws.scratch[:64], ws.status)
    with pytest.raises(ep.EPError):
        ep.ep_moe_decode(*c.dev, small)
    big = Case(600, 4, 2, 128, 128, seed=1)
    with pytest.raises(ep.EPError) as e:
        ep.ep_moe_decode(*big.dev)
    assert e.value.code == ep.EP_ERR_CAPACITY
    assert ep.ep_moe_decode(x[:0], idx[:0], w[:0], w13, s13, w2, s2).shape == (0, 256)
