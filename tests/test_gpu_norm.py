"""ep_rmsnorm against the formula in 64 bits.

Tolerances.  s = x + residual is one fp32 rounding of two bf16 numbers; the sum
of H squares is a tree and chains of positive terms, at most 64 roundings deep
for the sizes the kernel takes; mean, root, reciprocal and two products add 8.
So y is within 2^-17 of the formula (72 * 2^-24 < 2^-17), and its bf16 rounding
adds half a step.
"""
import pytest
import torch

from combine_expert_histogram_gb300 import binding as ep
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

REL = 2.0 ** -17
EPS = 1e-5


def make(T, H, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).bfloat16()
    r = (3 * torch.randn((T, H), generator=g)).bfloat16() if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).bfloat16()
    return x, r, w


def formula(x, r, w, eps=EPS):
    s = x.to(ref.F64) + (r.to(ref.F64) if r is not None else 0)
    return s, s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w.to(ref.F64)


def cuda(*ts):
    return [t.cuda() if t is not None else None for t in ts]


def check_scaled(rows, scales, y, quant, T, H):
    q = ref.decode(rows)
    noise = y.abs() * REL + 1e-37
    if quant == "mxfp8":
        b = ref.word_bytes(scales).to(ref.F64)
        amax = y.view(T, H // 32, 32).abs().amax(2)
        lo, hi = (torch.clamp(torch.floor(torch.log2(amax * (1 + k))) - 8, min=-127)
                  for k in (-REL, REL))
        assert ((b - 127 >= lo) & (b - 127 <= hi)).all()
        s = torch.exp2(b - 127).repeat_interleave(32, 1)
        r = y / s
        # half a step of E4M3 at the value; up to 512 saturates to 448
        step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(2.0 ** -6, 448.0))) - 3)
        over = (r.abs() - 448).clamp(min=0)
        assert ((q - r).abs() <= step / 2 + over + r.abs() * REL + 1e-30).all()
        return
    if quant == "fp8_f32":
        s = scales.cpu().to(ref.F64)
    else:
        words = ref.mn_to_rows(scales, T) if quant == "fp8_ue8m0_mn" else scales
        s = ref.ue8m0(words, H // 128)
        b = ref.word_bytes(words)
        assert (b[:, H // 128:] == 127).all()  # unused bytes of the last word
    lo, hi, s_lo, s_hi = ref.spread(y, noise, power=quant != "fp8_f32")
    assert ((s >= s_lo * (1 - ref.U)) & (s <= s_hi * (1 + ref.U))).all()
    v = q * ref.widen(s)
    slack = v.abs() * 4 * ref.U
    assert ((v >= lo - slack) & (v <= hi + slack)).all()


SHAPES = [(1, 128), (1, 7168), (3, 640), (17, 2048), (5, 1152), (2, 8192), (2, 8320), (3, 16384),
          (2, 32768), (257, 512)]


@pytest.mark.parametrize("quant", ["none", "fp8_f32", "fp8_ue8m0", "mxfp8", "fp8_ue8m0_mn"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_formula(T, H, quant):
    x, r, w = make(T, H, seed=H + T)
    s, y = formula(x, r, w)
    out, rows, scales, res = ep.ep_rmsnorm(*cuda(x, w), EPS, residual=r.cuda(), quant=quant)
    torch.cuda.synchronize()
    ref.close_bf16(out, y, y.abs() * REL)
    ref.close_bf16(res, s, s.abs() * ref.U)
    if quant != "none":
        check_scaled(rows, scales, y, quant, T, H)


def bytes_of(t):
    return t.cpu().view(torch.uint8)


@pytest.mark.parametrize("T", [3, 2500])
@pytest.mark.parametrize("quant", ["fp8_f32", "fp8_ue8m0", "mxfp8", "fp8_ue8m0_mn"])
def test_quantised_by_the_rule_of_dispatch(T, quant):
    """Rows of +-1 without eps have a mean square of 1, so y is +-weight, a bf16
    number: the 8-bit rows and scales are ep_dispatch's of the bf16 rows, bit for
    bit.  Among the weights are the groups whose quotient x / s is a tie of E4M3
    (or next to one) that a product by the rounded 1 / s moves."""
    H = 16384
    g = torch.Generator().manual_seed(T)
    w = ref.tie_groups(H // 128, g)
    w[40, 3], w[41, 5], w[42] = float("inf"), float("nan"), 0.0
    w[43, :3] = torch.tensor([3e38, -1e-39, 1e-30])
    w[44] *= 2.0 ** -130
    w[45] *= 2.0 ** 110
    w[46, 64:] = 0.0
    w = w.flatten().bfloat16().cuda()
    x = (torch.randint(0, 2, (T, H), generator=g) * 2 - 1).bfloat16().cuda()
    out, rows, scales, _ = ep.ep_rmsnorm(x, w, 0.0, quant=quant)
    assert torch.equal((x * w).view(torch.int16)[:, :40 * 128], out.view(torch.int16)[:, :40 * 128])
    L = ep.ep_layout(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1, align=1)
    want, want_s, _ = ep.ep_dispatch(L, out, quant)
    assert torch.equal(bytes_of(rows), bytes_of(want))
    if quant == "fp8_ue8m0_mn":
        scales, want_s = scales[:, :T].contiguous(), want_s[:, :T].contiguous()
    assert torch.equal(bytes_of(scales), bytes_of(want_s))
    if quant == "fp8_f32":
        q, s = ref.quantise_bf16(out.cpu()[:8, :40 * 128])
        assert torch.equal(ref.decode(rows[:8, :40 * 128]), q)
        assert torch.equal(scales.cpu()[:8, :40].to(ref.F64), s)


@pytest.mark.parametrize("H", [8, 24, 200, 2056, 4104])
def test_bf16_rows_of_any_multiple_of_8_without_residual(H):
    x, _, w = make(9, H, seed=H, residual=False)
    _, y = formula(x, None, w)
    out, rows, scales, res = ep.ep_rmsnorm(*cuda(x, w), EPS)
    assert rows is None and scales is None and res is None
    ref.close_bf16(out, y, y.abs() * REL)


@pytest.mark.parametrize("T", [700, 5000])
def test_many_rows(T):
    x, r, w = make(T, 1024, seed=T)
    s, y = formula(x, r, w)
    out, rows, scales, res = ep.ep_rmsnorm(*cuda(x, w), EPS, residual=r.cuda(), quant="fp8_f32")
    ref.close_bf16(out, y, y.abs() * REL)
    ref.close_bf16(res, s, s.abs() * ref.U)
    check_scaled(rows, scales, y, "fp8_f32", T, 1024)


def check_some_rows(T, H, quant, seed):
    """All bf16 rows against the formula on the device, 8-bit rows of some."""
    x, r, w = cuda(*make(T, H, seed=seed))
    out, rows, scales, res = ep.ep_rmsnorm(x, w, EPS, residual=r, quant=quant)
    s = x.to(ref.F64) + r.to(ref.F64)
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * w.to(ref.F64)
    assert ((res.to(ref.F64) - s).abs() <= s.abs() * (ref.BF16 + ref.U)).all()
    assert ((out.to(ref.F64) - y).abs() <= y.abs() * (ref.BF16 + 1.01 * REL) + 2.0 ** -133).all()
    if quant != "none":
        g = torch.Generator().manual_seed(seed)
        some = torch.cat([torch.tensor([0, T // 2, T - 1]), torch.randint(0, T, (20,), generator=g)])
        at = some.cuda()
        sc = scales[:, at] if quant == "fp8_ue8m0_mn" else scales[at]
        check_scaled(rows[at], sc, y[at].cpu(), quant, len(some), H)


@pytest.mark.parametrize("quant", ["none", "fp8_f32", "fp8_ue8m0", "mxfp8", "fp8_ue8m0_mn"])
@pytest.mark.parametrize("H", [2048, 2176, 4096, 4224, 7168, 8320, 32768])
def test_many_rows_of_two_and_four_vectors_a_lane(H, quant):
    """Blocks of many rows: lanes with one, two or four vectors, the last vectors of
    a row in all of them, in some warps, or in part of a warp."""
    check_some_rows(2500, H, quant, seed=H)


@pytest.mark.parametrize("quant", ["none", "fp8_f32", "fp8_ue8m0", "mxfp8", "fp8_ue8m0_mn"])
@pytest.mark.parametrize("H", [8320, 12416, 16512, 20608, 24704, 32640])
def test_few_long_rows(H, quant):
    """Few rows of two and four vectors a lane that end inside a vector's round."""
    check_some_rows(3, H, quant, seed=H)


@pytest.mark.parametrize("over", [-1, 0, 1])
@pytest.mark.parametrize("rows_per_sm", [1, 2, 3, 16])
def test_rows_around_multiples_of_the_processors(rows_per_sm, over):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check_some_rows(rows_per_sm * sms + over, 4224, "fp8_f32", seed=rows_per_sm)


@pytest.mark.parametrize("H", [2056, 4104, 8200, 16392])
def test_many_bf16_rows_of_any_multiple_of_8(H):
    check_some_rows(2500, H, "none", seed=H)


@pytest.mark.parametrize("quant", ["none", "fp8_f32", "mxfp8"])
def test_in_place(quant):
    """residual_out = residual and out = x give what separate buffers give."""
    x, r, w = make(33, 1280, seed=4)
    a = ep.ep_rmsnorm(*cuda(x, w), EPS, residual=r.cuda(), quant=quant)
    xd, rd, wd = cuda(x, r, w)
    b = ep.ep_rmsnorm(xd, wd, EPS, residual=rd, quant=quant, out=xd, residual_out=rd)
    for p, q in zip(a, b):
        assert p is None and q is None or torch.equal(p, q)


def test_8_bit_rows_alone():
    x, r, w = make(33, 1280, seed=5)
    a = ep.ep_rmsnorm(*cuda(x, w), EPS, residual=r.cuda(), quant="fp8_f32")
    b = ep.ep_rmsnorm(*cuda(x, w), EPS, residual=r.cuda(), quant="fp8_f32", with_out=False)
    assert b[0] is None
    for p, q in zip(a[1:], b[1:]):
        assert torch.equal(p, q)


def test_rows_of_zeros_and_large_values():
    """A zero row gives zeros (scale 1e-4 / 448, or the smallest of MX); rows near
    bf16's range square to finite fp32 sums as long as the formula's do."""
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    x[1] = 1e18
    x[2, 7] = 1e-20
    w = torch.ones(256, dtype=torch.bfloat16)
    for quant in ("fp8_f32", "fp8_ue8m0", "mxfp8"):
        out, rows, scales, _ = ep.ep_rmsnorm(*cuda(x, w), EPS, quant=quant)
        _, y = formula(x, None, w)
        ref.close_bf16(out, y, y.abs() * REL)
        assert (out[0] == 0).all() and (rows[0] == 0).all()
        if quant == "fp8_f32":
            want = torch.tensor(1e-4, dtype=torch.float32) / torch.tensor(448.0)
            assert (scales[0].cpu() == want).all()
        if quant == "mxfp8":
            assert (scales[0] == 0).all()


def test_a_row_of_nan_stays_in_its_row():
    x, r, w = make(4, 512, seed=8)
    x[2, 100] = float("nan")
    x[3, 5] = float("inf")
    out, rows, scales, _ = ep.ep_rmsnorm(*cuda(x, w), EPS, residual=r.cuda(), quant="fp8_f32")
    _, y = formula(x, r, w)
    ref.close_bf16(out[:2], y[:2], y[:2].abs() * REL)
    check_scaled(rows[:2], scales[:2], y[:2], "fp8_f32", 2, 512)
    assert out[2].isnan().all()


def test_no_rows_and_refusals():
    x, r, w = cuda(*make(0, 256))
    out, rows, scales, res = ep.ep_rmsnorm(x, w, EPS, residual=r, quant="fp8_f32")
    assert out.shape == (0, 256) and rows.shape == (0, 256)
    x, r, w = cuda(*make(4, 256))
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x.float(), w)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, w[:128])
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x.t(), w)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, w, residual=r.cpu())
    with pytest.raises(ep.EPError):
        ep.ep_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(ep.EPError):
        ep.ep_rmsnorm(x, w, eps=float("nan"))
    with pytest.raises(ep.EPError):
        ep.ep_rmsnorm(x, w, with_out=False)
    with pytest.raises(ep.EPError):  # no multiple of 128
        ep.ep_rmsnorm(x[:, :136].contiguous(), w[:136].contiguous(), quant="fp8_f32")


def test_another_stream_and_a_replayed_graph():
    x, r, w = make(6, 1024, seed=11)
    xd, rd, wd = cuda(x, r, w)
    s = torch.cuda.Stream()
    out = torch.empty_like(xd)
    res = torch.empty_like(xd)
    with torch.cuda.stream(s):
        ep.ep_rmsnorm(xd, wd, EPS, residual=rd, out=out, residual_out=res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.ep_rmsnorm(xd, wd, EPS, residual=rd, out=out, residual_out=res, stream=s)
    for seed in (12, 13):
        x, r, _ = make(6, 1024, seed=seed)
        xd.copy_(x)
        rd.copy_(r)
        g.replay()
        torch.cuda.synchronize()
        _, y = formula(x, r, w)
        ref.close_bf16(out, y, y.abs() * REL)


@pytest.mark.parametrize("T", [3, 600])
def test_norm_straight_into_dispatch(T):
    """ep_dispatch directly after the norm (its early reads of x included): the
    rows it writes are its own quantisation of the norm's bf16 rows."""
    E, K, H = 16, 4, 512
    x, r, w = make(T, H, seed=T)
    xd, rd, wd = cuda(x, r, w)
    idx = torch.stack([torch.randperm(E)[:K] for _ in range(T)]).to(torch.int32).cuda()
    L = ep.ep_layout(idx, E)
    torch.cuda.synchronize()
    out, _, _, _ = ep.ep_rmsnorm(xd, wd, EPS, residual=rd)
    rows, scales, _ = ep.ep_dispatch(L, out, "fp8_f32")
    torch.cuda.synchronize()
    q, s = ref.quantise_bf16(out.cpu())
    dst = L.dst_row.cpu().long()[:T * K]
    assert torch.equal(ref.decode(rows[dst.cuda()]), q.repeat_interleave(K, 0))
    assert torch.equal(scales.cpu()[dst].to(ref.F64), s.repeat_interleave(K, 0))


def test_weight_that_the_kernel_before_writes():
    """combine lets the norm start early, and its last row is the norm's weight: the
    norm has to wait for it.  The stream is held, so that the launches queue."""
    T, K, E, H = 1024, 32, 64, 1024
    g = torch.Generator().manual_seed(12)
    idx = torch.rand((T, E), generator=g).topk(K).indices.int().cuda()
    w = torch.rand((T, K), generator=g).cuda()
    L = ep.ep_layout(idx, E)
    ys = [torch.randn((ep.ep_rows_capacity(L), H), generator=g).bfloat16().cuda() for _ in range(2)]
    x = torch.randn((8, H), generator=g).bfloat16().cuda()
    want = []
    for y in ys:
        weight = ep.ep_combine(L, y, w)[-1].clone()
        torch.cuda.synchronize()
        want.append(ep.ep_rmsnorm(x, weight, EPS)[0])
    out = ep.ep_combine(L, ys[1], w)
    big = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    for _ in range(6):
        big.fill_(1)
    got = []
    for i in range(20):
        ep.ep_combine(L, ys[i % 2], w, out=out)
        got.append(ep.ep_rmsnorm(x, out[-1], EPS)[0])
    torch.cuda.synchronize()
    for i, h in enumerate(got):
        assert torch.equal(h, want[i % 2]), i
