"""ep_kv_append, ep_attn_decode and ep_attn_prefill against their formulas in 64 bits."""
import pytest
import torch

from combine_expert_histogram_gb300 import binding as ep
from tests import layer_ref as ref
from tests.attn_ref import Seqs, close, in_8_bits, rotate

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF, F8 = "none", "fp8_ue8m0"


def angles(positions, R, seed=0):
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def poisoned(T, Hq, D):
    """An output whose every element is seen to be written or not."""
    return torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")


# ---------------------------------------------------------------------- append
def check_append(s, R, inter=False, with_q=True, in_place=False, fused=True):
    """Append s's newest tokens to its cache, from which they are first taken out."""
    T, Hkv, D = s.T, s.Hkv, s.D
    cs = angles(max(s.lens + [1]), max(R, 2))
    if fused:  # columns of one projection
        qkv = torch.randn((T, s.Hq + 2 * Hkv, D), generator=s.g).bfloat16()
        q, k, v = qkv[:, :s.Hq], qkv[:, s.Hq:s.Hq + Hkv], qkv[:, s.Hq + Hkv:]
        d = qkv.cuda()
        dq, dk, dv = d[:, :s.Hq], d[:, s.Hq:s.Hq + Hkv], d[:, s.Hq + Hkv:]
    else:
        q, k, v = (torch.randn((T, n, D), generator=s.g).bfloat16() for n in (s.Hq, Hkv, Hkv))
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    cache, seqs, _ = s.cuda()
    before = [t.clone() for t in (cache.k, cache.v)]
    scales = [t.clone() for t in (cache.k_scales, cache.v_scales)] if s.quant == F8 else None
    out = dq if in_place else poisoned(T, s.Hq, D)
    was = out.clone()
    got = ep.ep_kv_append(cache, seqs, dk, dv, cos_sin=cs.cuda() if R else None,
                          q=dq if with_q else None, q_out=out if with_q else None,
                          interleaved=inter)
    torch.cuda.synchronize()
    seqs.check_status()
    pos, own, place = [], [], []
    starts = s.starts if s.new is not None else list(range(len(s.lens) + 1))
    for b, L in enumerate(s.lens):
        n = starts[b + 1] - starts[b]
        for r in range(n):
            i = L - n + r
            if i >= 0:
                own.append(starts[b] + r)
                pos.append(i)
                place.append((int(s.table[b, i // s.page]), i % s.page))
    c, n = (x[pos] for x in cs.chunk(2, 1))
    own_t = torch.tensor(own, dtype=torch.long)
    turn = (lambda x: rotate(x, c, n, inter)) if R else (lambda x: x)
    if with_q:
        want = was.cpu()
        want[own_t] = turn(q[own_t].to(ref.F64)).float().bfloat16()
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    page, row = (torch.tensor([p[x] for p in place], dtype=torch.long) for x in (0, 1))
    for x, f, old, now, sc in ((k, turn, before[0], cache.k, 0), (v, lambda y: y, before[1], cache.v, 1)):
        y = f(x[own_t].to(ref.F64))
        want = old.cpu()
        if s.quant == BF:
            want[page, row] = y.float().bfloat16()
            assert torch.equal(now.cpu().view(torch.int16), want.view(torch.int16))
            continue
        q8, e = in_8_bits(y)
        want[page, row] = q8.float().to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(now.cpu(), want)
        es = scales[sc].cpu()
        es[page, :, row] = e
        assert torch.equal((cache.k_scales, cache.v_scales)[sc].cpu(), es)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 64, False), (128, 128, True),
                                       (64, 64, False), (64, 16, False), (64, 32, True),
                                       (128, 16, True), (64, 0, False), (128, 0, False),
                                       (128, 112, False), (64, 48, True)])
def test_append_rotations(D, R, inter, quant):
    check_append(Seqs([5, 40, 17], [5, 3, 1], D=D, quant=quant, Hq=5, Hkv=5, page=8), R, inter)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("lens,new,kw", [
    ([1], None, {}),
    ([4001], None, dict(page=64, Hq=32, Hkv=4)),
    ([9, 0, 3, 0, 70], None, {}),                      # rows of a padded batch: skipped
    ([70], [70], dict(page=24)),
    ([0, 30, 0], [0, 7, 0], {}),
    ([3, 20], [5, 20], {}),                            # more rows than tokens: skipped
    ([33, 64, 100], [33, 1, 99], dict(gap=3, tail=4)),  # rows that no sequence owns
    ([600, 500], [600, 400], dict(page=128, Hq=7, Hkv=1)),
    ([900], [900], dict(page=128, Hq=16, Hkv=8)),      # 3 million values: a fused product shows
    ([17, 9], [17, 2], dict(layout="rows")),
    ([17, 9], [17, 2], dict(layout="slice", D=64)),
])
def test_append_sequences(lens, new, kw, quant):
    kw = {"Hq": 6, "Hkv": 3, **kw}
    check_append(Seqs(lens, new, quant=quant, **kw), 64)


@pytest.mark.parametrize("kw", [dict(with_q=False), dict(in_place=True), dict(fused=False)])
def test_append_forms(kw):
    check_append(Seqs([20, 300], [20, 11], Hq=8, Hkv=2), 128, **kw)


@pytest.mark.parametrize("D", [64, 128])
def test_append_rows_that_are_not_finite(D):
    """A row with an infinity or a NaN is stored as NaN, its neighbours as ever; the largest
    and the smallest values have their scales."""
    s = Seqs([6], [6], Hq=1, Hkv=1, D=D, page=8, quant=F8)
    k = torch.randn((6, 1, D), generator=s.g)
    k[1, 0, 3], k[2, 0, D - 1], k[3, 0] = float("inf"), float("nan"), 3.0e38
    k[4, 0], k[5, 0] = 0.0, 1e-30
    k = k.bfloat16()
    cache, seqs, _ = s.cuda()
    ep.ep_kv_append(cache, seqs, k.cuda(), k.cuda())
    seqs.check_status()
    val = torch.ldexp(ref.decode(cache.k), cache.k_scales.cpu().transpose(1, 2)[..., None].int() - 127)
    val[cache.k_scales.cpu().transpose(1, 2) == 255] = float("nan")
    at = s.table[0, 0].long()
    got = val[at, :6, 0]
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
    assert cache.k_scales.cpu()[at, 0, 1:3].tolist() == [255, 255]
    fine = [0, 3, 4, 5]
    q8, e = in_8_bits(k[fine, 0].to(ref.F64))
    assert torch.equal(got[fine], torch.ldexp(q8, e[:, None].int() - 127))
    assert torch.equal(cache.k, cache.v) and torch.equal(cache.k_scales, cache.v_scales)


def test_append_bad_pages_and_positions():
    s = Seqs([10, 20, 30], [2, 2, 2], Hq=2, Hkv=1, page=8)
    k = torch.ones((6, 1, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((6, 2, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (-1, s.pages, 1 << 30, -(1 << 31)):
        cache, seqs, _ = s.cuda()
        seqs.block_table[1, 2] = bad
        before = cache.k.clone()
        ep.ep_kv_append(cache, seqs, k, k)
        with pytest.raises(ep.EPError) as e:
            seqs.check_status()
        assert e.value.code == ep.EP_ERR_BAD_PAGE
        changed = (cache.k.view(torch.int16) != before.view(torch.int16)).any(-1).any(-1).cpu()
        want = torch.zeros_like(changed)
        for b, i in ((0, 8), (0, 9), (2, 28), (2, 29)):
            want[s.table[b, i // 8].long(), i % 8] = True
        assert torch.equal(changed, want)  # sequence 1's two tokens, at 18 and 19, are skipped
    cache, seqs, _ = s.cuda()  # a table of 20 positions: sequence 2's are past it
    out = poisoned(6, 2, 128)
    ep.ep_kv_append(cache, seqs, k, k, cos_sin=angles(20, 32).cuda(), q=q, q_out=out)
    with pytest.raises(ep.EPError):
        seqs.check_status()
    assert torch.isnan(out[4:]).all() and not torch.isnan(out[:4]).any()
    cache, seqs, _ = s.cuda()  # a length past the block table
    seqs.kv_len[1] = 1000
    ep.ep_kv_append(cache, seqs, k, k)
    with pytest.raises(ep.EPError):
        seqs.check_status()


# ------------------------------------------------------------------- attention
def run(s, decode, **kw):
    cache, seqs, q = s.cuda()
    out = poisoned(s.T, s.Hq, s.D)
    lse = torch.full((s.T, s.Hq), 7.0, device="cuda")
    f = ep.ep_attn_decode if decode else ep.ep_attn_prefill
    assert f(cache, seqs, q, out=out, lse=lse, **kw) is out
    torch.cuda.synchronize()
    seqs.check_status()
    own = s.owned()
    assert torch.isnan(out.cpu()[~own]).all() and (lse.cpu()[~own] == 7.0).all()
    return out, lse


def check(s, decode, **kw):
    out, lse = run(s, decode, **kw)
    close(s, out, lse, **kw)


HEADS = [(1, 1), (4, 4), (4, 2), (8, 1), (15, 3), (16, 1), (34, 2), (64, 1)]


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_decode_heads(Hq, Hkv, D, quant):
    check(Seqs([100, 1, 33], Hq=Hq, Hkv=Hkv, D=D, quant=quant), True)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("lens,kw", [
    ([1], {}), ([2], {}), ([7], dict(page=8)), ([8], dict(page=8)), ([15, 16, 17], dict(page=24)),
    ([0], {}), ([0, 5, 0, 0, 9, 0], {}), ([127, 128, 129, 255, 256, 257], dict(page=64)),
    ([1000, 10, 1, 500, 3], dict(page=128)), ([5000], dict(page=16, Hq=8, Hkv=1)),
    ([4097], dict(page=64, Hq=32, Hkv=4)), (list(range(40)), dict(page=8, D=64)),
    ([300, 20], dict(layout="rows")), ([300, 20], dict(layout="slice")),
    ([777, 31], dict(layout="slice", D=64, page=40)), ([20000, 3, 7000], dict(page=256, Hq=2, Hkv=1)),
])
def test_decode_lengths(lens, kw, quant):
    check(Seqs(lens, quant=quant, **kw), True)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 3), (100, 64), (1000, 4),
                                          (128, 128), (5, 2000), (1 << 30, 1 << 30)])
def test_decode_window(window, sinks, quant):
    s = Seqs([0, 1, 5, 16, 17, 130, 1500], page=16, quant=quant)
    # pages that no visible key is in may be gone
    for b, L in enumerate(s.lens):
        for e in range(-(-L // 16)):
            if 16 * e >= sinks and 16 * e + 15 <= L - 1 - window:
                s.table[b, e] = -1
    want = Seqs([0, 1, 5, 16, 17, 130, 1500], page=16, quant=quant)
    out, lse = run(s, True, window=window, sinks=sinks)
    close(want, out, lse, window=window, sinks=sinks)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (0.01, 1.0), (0.088, 8.0), (1e-30, 1.0)])
def test_scales(scale, spread, decode):
    s = Seqs([200, 30], None if decode else [40, 30], spread=spread)
    check(s, decode, scale=scale)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_prefill_heads(Hq, Hkv, D, quant):
    check(Seqs([100, 1, 33], [60, 1, 33], Hq=Hq, Hkv=Hkv, D=D, quant=quant), False)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("lens,new,kw", [
    ([1], [1], {}), ([2], [2], {}), ([9], [9], dict(page=8)), ([0], [0], {}), ([3], [0], {}),
    ([0, 5, 0], [0, 5, 0], {}), ([3, 4], [7, 4], {}),  # rows before the first key: empty
    ([127, 128, 129], [127, 128, 129], dict(page=64)), ([255, 256, 257], [1, 2, 3], dict(page=24)),
    ([700], [700], dict(page=128)), ([1300], [5], dict(page=8)), ([600, 40], [300, 40], dict(Hq=8, Hkv=1)),
    ([50, 60, 70], [10, 20, 30], dict(gap=2, tail=5)), ([300, 20], [129, 20], dict(layout="rows")),
    ([300, 20], [100, 20], dict(layout="slice")), ([777, 31], [77, 3], dict(layout="slice", D=64, page=40)),
    (list(range(1, 30)), [min(3, n) for n in range(1, 30)], dict(page=8, D=64)),
    ([520], None, {}), ([12, 0, 300], None, dict(Hq=2, Hkv=2)), ([513], [513], dict(Hq=1, Hkv=1, D=64)),
])
def test_prefill_lengths(lens, new, kw, quant):
    check(Seqs(lens, new, quant=quant, **kw), False)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 3), (100, 64), (300, 4),
                                          (128, 128), (5, 2000), (1 << 30, 1 << 30)])
def test_prefill_window(window, sinks, quant):
    def make():
        return Seqs([1, 5, 130, 700, 600], [1, 5, 100, 700, 9], page=16, quant=quant, Hq=4, Hkv=2)
    s = make()
    for b, L in enumerate(s.lens):
        for e in range(-(-L // 16)):
            if 16 * e >= sinks and 16 * e + 15 <= L - s.new[b] - window:
                s.table[b, e] = -1
    out, lse = run(s, False, window=window, sinks=sinks)
    close(make(), out, lse, window=window, sinks=sinks)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,new,Hq,Hkv,kw", [
    ([4000], [3], 8, 1, {}), ([4000, 1, 2100], [2, 1, 40], 4, 2, {}), ([1500], [300], 8, 1, {}),
    ([3000, 700], [130, 5], 2, 2, dict(window=900, sinks=200)), ([256], [1], 1, 1, {}),
    ([257, 600, 0], [2, 0, 0], 6, 1, {}),
])
def test_prefill_few_tokens(lens, new, Hq, Hkv, kw, D, quant):
    """Keys shared out among blocks, and not."""
    s = Seqs(lens, new, Hq=Hq, Hkv=Hkv, D=D, quant=quant, page=64, tail=2)
    out, lse = run(s, False, **kw)
    close(s, out, lse, **kw)
    cache, seqs, q = s.cuda()
    n = ep.ep_attn_prefill_workspace_bytes(s.T, len(lens), Hq, Hkv, D)
    assert n > 0
    dirty = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    own = s.owned()
    again = ep.ep_attn_prefill(cache, seqs, q, scratch=dirty, **kw)
    assert torch.equal(again.cpu()[own], out.cpu()[own])
    lib = ep.load_library()
    alone = poisoned(s.T, Hq, D)
    import ctypes
    code = lib.ep_attn_prefill(ctypes.byref(cache._c), ctypes.byref(seqs._struct(s.T)), q.data_ptr(),
                               Hq * D, Hq, D ** -0.5, kw.get("window", 0), kw.get("sinks", 0),
                               alone.data_ptr(), None, None, 0, None)
    assert code == 0
    torch.cuda.synchronize()
    close(s, alone, **kw)
    with pytest.raises(ep.EPError):
        ep.ep_attn_prefill(cache, seqs, q, scratch=dirty[:n - 16].clone(), **kw)


@pytest.mark.parametrize("decode", [True, False])
def test_long_sequences(decode):
    """A cache of more than 2^32 bytes, with the sequence's pages at both of its ends."""
    page, D, n = 64, 128, 3000
    used = -(-n // page)
    pages = 320_000  # 5.2 GB each of keys and values
    small = Seqs([n], None if decode else [150], Hq=2, Hkv=1, D=D, page=page, spare=0, extra_cols=0)
    k, v = (torch.zeros((pages, 1, page, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
            for _ in range(2))
    to = torch.tensor([pages - 1 - e if e % 2 else e for e in range(used)])
    at = small.table[0].long()
    for dst, src in ((k, small.k), (v, small.v)):
        dst[to.cuda()] = src[at].cuda()
    cache = ep.KvCache(k, v)
    _, seqs, q = small.cuda()
    seqs.block_table[0] = to.to(torch.int32).cuda()
    f = ep.ep_attn_decode if decode else ep.ep_attn_prefill
    out = f(cache, seqs, q)
    seqs.check_status()
    close(small, out)
    new = torch.randn((small.T, 1, D), generator=small.g).bfloat16().cuda()
    ep.ep_kv_append(cache, seqs, new, new)
    assert torch.equal(k[to[-1], (n - 1) % page, 0], new[-1, 0])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 256])
def test_prefill_page_sizes(page, quant, D):
    """Whole row blocks and row blocks of few rows, one after another, over pages of every kind."""
    lens = [1500, 200, 1300, 3, 900]
    s = Seqs(lens, [700, 3, 1, 3, 33], Hq=16, Hkv=2, D=D, page=page, quant=quant)
    check(s, False)
    out, _ = run(s, False)
    again, _ = run(s, False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("what", ["k", "v"])
def test_prefill_not_finite_in_later_keys(what, quant):
    """A key or value that is not a number: rows before it do not see it, later ones are NaN."""
    s = Seqs([300], [300], Hq=4, Hkv=2, quant=quant)
    for j in (130, 131, 250):
        p, r = s.table[0, j // s.page].long(), j % s.page
        if quant == BF:
            getattr(s, what)[p, r, 0, 5] = float("nan")
        else:
            getattr(s, what + "s")[p, 0, r] = 255
    out, lse = run(s, False)
    clean = Seqs([300], [300], Hq=4, Hkv=2, quant=quant)
    want, noise, want_l, noise_l = clean.attention()
    if what == "v":  # the sum of probabilities is without the values
        assert ((lse.cpu().to(ref.F64) - want_l).abs() <= noise_l).all()
    ref.close_bf16(out[:130].cpu(), want[:130], noise[:130])
    ref.close_bf16(out[:, 2:].cpu(), want[:, 2:], noise[:, 2:])  # the other key head's queries
    hit = out[130:, :2].cpu()
    if what == "v" and quant == BF:
        assert torch.isnan(hit[..., 5]).all()
        rest = [d for d in range(128) if d != 5]
        ref.close_bf16(hit[..., rest], want[130:, :2][..., rest], noise[130:, :2][..., rest])
    else:
        assert torch.isnan(hit).all()


@pytest.mark.parametrize("quant", [BF, F8])
def test_prefill_not_finite_outside_the_window(quant):
    """Values that fell out of a row's window, and infinities among them, do not reach it."""
    s = Seqs([400], [400], Hq=2, Hkv=1, quant=quant)
    for j in (7, 150):
        p, r = s.table[0, j // s.page].long(), j % s.page
        if quant == BF:
            s.v[p, r, 0, 9] = float("inf")
            s.k[p, r, 0, 3] = float("nan")
        else:
            s.vs[p, 0, r] = 255
    out, _ = run(s, False, window=20, sinks=2)
    want, noise, _, _ = Seqs([400], [400], Hq=2, Hkv=1, quant=quant).attention(window=20, sinks=2)
    i = torch.arange(400)
    seen = ((i >= 7) & (i < 27)) | ((i >= 150) & (i < 170))
    ref.close_bf16(out.cpu()[~seen], want[~seen], noise[~seen])
    assert torch.isnan(out.cpu()[seen]).any(-1).all()


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("what", ["k", "v"])
def test_decode_not_finite_in_seen_keys(what, quant):
    """A key or value that is not a number makes every query head that sees it NaN, whatever the
    sign of its product with the query."""
    s = Seqs([300, 40, 5], None, Hq=32, Hkv=2, quant=quant, page=64)
    for j in (3, 250):  # behind the second sequence's last key lies what its page holds
        p, r = s.table[0, j // s.page].long(), j % s.page
        if quant == BF:
            getattr(s, what)[p, r, 0, 5] = float("nan")
        else:
            getattr(s, what + "s")[p, 0, r] = 255
    out, lse = run(s, True)
    clean = Seqs([300, 40, 5], None, Hq=32, Hkv=2, quant=quant, page=64)
    want, noise, want_l, noise_l = clean.attention()
    ref.close_bf16(out[1:].cpu(), want[1:], noise[1:])
    ref.close_bf16(out[:1, 16:].cpu(), want[:1, 16:], noise[:1, 16:])
    hit = out[0, :16].cpu()
    if what == "v" and quant == BF:
        assert torch.isnan(hit[:, 5]).all()
        rest = [d for d in range(128) if d != 5]
        ref.close_bf16(hit[:, rest], want[0, :16][:, rest], noise[0, :16][:, rest])
    else:
        assert torch.isnan(hit).all()
    if what == "v":
        assert ((lse.cpu().to(ref.F64) - want_l).abs() <= noise_l).all()


def test_infinite_value_that_is_seen():
    """An infinite value channel is infinite in every row that sees it, the others are not."""
    s = Seqs([200], [200], Hq=2, Hkv=1)
    p, r = s.table[0, 150 // s.page].long(), 150 % s.page
    s.v[p, r, 0, 9] = float("-inf")
    out, _ = run(s, False)
    got = out.cpu()
    assert (got[150:, :, 9] == float("-inf")).all() and torch.isfinite(got[:150]).all()
    assert torch.isfinite(got[150:, :, :9]).all() and torch.isfinite(got[150:, :, 10:]).all()


def test_decode_not_finite_outside_the_window():
    s = Seqs([400, 90], Hq=4, Hkv=2)
    for b, j in ((0, 300), (0, 2), (1, 60)):
        p, r = s.table[b, j // s.page].long(), j % s.page
        s.v[p, r], s.k[p, r] = float("inf"), float("nan")
    out, lse = run(s, True, window=20, sinks=2)
    close(Seqs([400, 90], Hq=4, Hkv=2), out, lse, window=20, sinks=2)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("quant", [BF, F8])
def test_bad_pages(quant, decode):
    """A needed page that the cache has not: the status says so, other sequences are right."""
    s = Seqs([100, 90, 80], None if decode else [20, 90, 3], quant=quant)
    want, noise, _, _ = s.attention()
    t0, t1 = (1, 2) if decode else (20, 110)
    for bad in (-1, s.pages, 1 << 30, -(1 << 31)):
        cache, seqs, q = s.cuda()
        seqs.block_table[1, 2] = bad
        f = ep.ep_attn_decode if decode else ep.ep_attn_prefill
        out = f(cache, seqs, q).cpu()
        with pytest.raises(ep.EPError) as e:
            seqs.check_status()
        assert e.value.code == ep.EP_ERR_BAD_PAGE
        other = [t for t in range(s.T) if not t0 <= t < t1]
        ref.close_bf16(out[other], want[other], noise[other])
        assert torch.isfinite(out).all()  # its rows count as zeros
    cache, seqs, q = s.cuda()
    seqs.kv_len[1] = 1 << 30
    f(cache, seqs, q)
    with pytest.raises(ep.EPError):
        seqs.check_status()


@pytest.mark.parametrize("decode", [True, False])
def test_sequence_lists_that_are_none(decode):
    """Negative lengths, falling and far starts: no access outside the arrays."""
    s = Seqs([30, 40, 50], None if decode else [3, 4, 5])
    cache, seqs, q = s.cuda()
    f = ep.ep_attn_decode if decode else ep.ep_attn_prefill
    seqs.kv_len[1] = -5
    out = f(cache, seqs, q)
    assert (out[1] == 0).all() if decode else (out[3:7] == 0).all()
    if not decode:
        new = torch.zeros((s.T, s.Hkv, s.D), dtype=torch.bfloat16, device="cuda")
        for starts in ([9, 3, 7, 1], [-4, 5, 6, 12], [0, 1 << 30, 4, 12], [0, 4, 8, 1 << 30],
                       [12, 12, 12, 12], [-(1 << 31), (1 << 31) - 1, 0, 5]):
            seqs.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
            f(cache, seqs, q)
            ep.ep_kv_append(cache, seqs, new, new)
    torch.cuda.synchronize()


@pytest.mark.parametrize("decode", [True, False])
def test_strided_queries_and_out_of_place(decode):
    s = Seqs([300, 4], None if decode else [17, 4], Hq=6, Hkv=2)
    cache, seqs, q = s.cuda()
    wide = torch.full((s.T, 10, s.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = q
    f = ep.ep_attn_decode if decode else ep.ep_attn_prefill
    assert torch.equal(f(cache, seqs, wide[:, 2:8]), f(cache, seqs, q))
    with pytest.raises(ValueError):
        f(cache, seqs, q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError):
        f(cache, seqs, q.float())
    with pytest.raises(ValueError):
        f(cache, seqs, q, out=q.float())
    with pytest.raises(ep.EPError):
        f(cache, seqs, q[:, :5].contiguous())  # no multiple of the key heads


@pytest.mark.parametrize("quant", [BF, F8])
def test_same_call_same_bits(quant):
    s = Seqs([3000, 17, 800, 2500], quant=quant, Hq=16, Hkv=2, page=32)
    cache, seqs, q = s.cuda()
    ws = ep.new_attn_workspace(4, 16, 2, 128)
    first = ep.ep_attn_decode(cache, seqs, q, workspace=ws)
    for _ in range(20):
        assert torch.equal(ep.ep_attn_decode(cache, seqs, q, workspace=ws), first)
    for _ in range(3):
        assert torch.equal(ep.ep_attn_decode(cache, seqs, q), first)
    p = Seqs([900, 300], [500, 300], quant=quant)
    cache, seqs, q = p.cuda()
    first = ep.ep_attn_prefill(cache, seqs, q)
    for _ in range(20):
        assert torch.equal(ep.ep_attn_prefill(cache, seqs, q), first)


def test_one_workspace_for_smaller_batches():
    ws = ep.new_attn_workspace(50, 16, 2, 128)
    for lens in ([10000], [5] * 50, [4000, 1, 900], list(range(0, 500, 10))):
        s = Seqs(lens, Hq=16, Hkv=2, page=32)
        cache, seqs, q = s.cuda()
        out = ep.ep_attn_decode(cache, seqs, q, workspace=ws)
        seqs.check_status()
        close(s, out)


def test_workspace_that_was_not_zeros():
    s = Seqs([5000], Hq=2, Hkv=1)
    cache, seqs, q = s.cuda()
    ws = ep.new_attn_workspace(1, 2, 1, 128)
    ws.scratch.fill_(0xFF)
    ep.ep_attn_decode(cache, seqs, q, workspace=ws)
    with pytest.raises(ep.EPError) as e:
        seqs.check_status()
    assert e.value.code == ep.EP_ERR_INVALID_ARG


def test_workspace_too_small():
    s = Seqs([100])
    cache, seqs, q = s.cuda()
    with pytest.raises(ep.EPError):
        ep.ep_attn_decode(cache, seqs, q, workspace=ep.AttnWorkspace(
            torch.empty(8, dtype=torch.uint8, device="cuda")))


@pytest.mark.parametrize("B", [1500, 5000])
def test_many_sequences(B):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    check(Seqs(lens, Hq=2, Hkv=1, D=64, page=8), True)
    new = [min(n, int(m)) for n, m in zip(lens, torch.randint(0, 4, (B,), generator=g))]
    check(Seqs(lens, new, Hq=2, Hkv=1, D=64, page=8), False)


@pytest.mark.parametrize("quant", [BF, F8])
def test_replayed_graph_follows_the_arrays(quant):
    """append and decode captured once; lengths, tables and tokens change between replays."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    lens = [40, 1, 300]
    s = Seqs([n + 3 for n in lens], Hq=Hq, Hkv=Hkv, D=D, page=page, quant=quant)
    cache, seqs, _ = s.cuda()
    cs = angles(400, D)
    dcs = cs.cuda()
    k, v = (torch.zeros((3, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, rot, out = (torch.zeros((3, Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ws = ep.new_attn_workspace(3, Hq, Hkv, D)

    def step():
        ep.ep_kv_append(cache, seqs, k, v, cos_sin=dcs, q=q, q_out=rot)
        ep.ep_attn_decode(cache, seqs, rot, workspace=ws, out=out, window=100, sinks=3)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    for _ in range(2):  # two graphs share the workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
    for t in range(3):
        now = [n + t + 1 for n in lens]
        seqs.kv_len.copy_(torch.tensor(now, dtype=torch.int32))
        nk, nv, nq = (torch.randn((3, n, D), generator=s.g).bfloat16() for n in (Hkv, Hkv, Hq))
        k.copy_(nk), v.copy_(nv), q.copy_(nq)
        graphs[t % 2].replay()
        torch.cuda.synchronize()
        seqs.check_status()
        pos = [n - 1 for n in now]
        c, sn = (x[pos] for x in cs.chunk(2, 1))
        s.lens = now
        s.q = rotate(nq.to(ref.F64), c, sn, False).float().bfloat16()
        yk = rotate(nk.to(ref.F64), c, sn, False)
        for b, i in enumerate(pos):
            at = (s.table[b, i // page].long(), i % page)
            for val, y in ((s.kval, yk[b]), (s.vval, nv[b].to(ref.F64))):
                if quant == BF:
                    val[at] = y.float().bfloat16().to(ref.F64)
                else:
                    q8, e = in_8_bits(y)
                    val[at] = torch.ldexp(q8, e[:, None].int() - 127)
        close(s, out, window=100, sinks=3)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
def test_replayed_prompts_follow_the_arrays(quant, D):
    """Prompts' attention captured twice over one scratch; lengths and rows' owners change between
    replays, down to nothing."""
    s = Seqs([700, 90, 400], [300, 90, 7], Hq=8, Hkv=2, D=D, quant=quant)
    cache, seqs, q = s.cuda()
    n = ep.ep_attn_prefill_workspace_bytes(s.T, 3, 8, 2, D)
    scratch = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = poisoned(s.T, 8, D), torch.empty((s.T, 8), device="cuda")

    def step():
        ep.ep_attn_prefill(cache, seqs, q, out=out, lse=lse, scratch=scratch, window=150, sinks=20)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
    for x, (lens, new) in enumerate([([700, 90, 400], [300, 90, 7]), ([650, 40, 0], [1, 40, 0]),
                                     ([0, 0, 0], [0, 0, 0]), ([300, 90, 399], [300, 1, 96])]):
        s.lens, s.new, s.starts = lens, new, [0]
        for m in new:
            s.starts.append(s.starts[-1] + m)
        seqs.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        seqs.q_start.copy_(torch.tensor(s.starts, dtype=torch.int32))
        out.fill_(float("nan"))
        graphs[x % 2].replay()
        torch.cuda.synchronize()
        seqs.check_status()
        own = s.owned()
        assert torch.isnan(out.cpu()[~own]).all()
        close(s, out, lse, window=150, sinks=20)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("quant", [BF, F8])
def test_largest_heads_and_pages(quant, decode):
    """The most query heads on one key head; the largest pages, the last one hardly used."""
    lens = [130, 3]
    check(Seqs(lens, None if decode else [5, 3], Hq=1024, Hkv=1, quant=quant, D=64), decode)
    lens = [4097, 4000]
    check(Seqs(lens, None if decode else [300, 1], Hq=4, Hkv=2, quant=quant, page=4096), decode)


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("layout", ["heads", "rows"])
def test_a_prompt_its_next_chunk_and_single_tokens(quant, layout):
    """The run of a model's layer: append and attend a prompt in two chunks, then token by token."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    total, cuts = [150, 61], [(100, 40), (45, 18), (1, 1), (1, 1), (3, 1)]
    s = Seqs(total, [1, 1], Hq=Hq, Hkv=Hkv, D=D, page=page, quant=quant, layout=layout)
    cache, handle, _ = s.cuda()
    cs = angles(200, D)
    have = [0, 0]
    for new in cuts:
        have = [h + n for h, n in zip(have, new)]
        T = sum(new)
        s.lens, s.new, s.T = list(have), list(new), T
        s.starts = [0, new[0], T]
        single = new == (1, 1)
        seqs = ep.new_kv_seqs(handle.block_table, torch.tensor(have, dtype=torch.int32).cuda(),
                              None if single else torch.tensor(s.starts, dtype=torch.int32).cuda())
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=s.g).bfloat16()
        d = qkv.cuda()
        q = ep.ep_kv_append(cache, seqs, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], cos_sin=cs.cuda(),
                            q=d[:, :Hq])
        out = (ep.ep_attn_decode if single else ep.ep_attn_prefill)(cache, seqs, q)
        torch.cuda.synchronize()
        seqs.check_status()
        pos = [h - n + r for h, n in zip(have, new) for r in range(n)]
        b = [x for x, n in enumerate(new) for _ in range(n)]
        c, sn = (x[pos] for x in cs.chunk(2, 1))
        s.q = rotate(qkv[:, :Hq].to(ref.F64), c, sn, False).float().bfloat16()
        yk = rotate(qkv[:, Hq:Hq + Hkv].to(ref.F64), c, sn, False)
        for t in range(T):
            at = (s.table[b[t], pos[t] // page].long(), pos[t] % page)
            for val, y in ((s.kval, yk[t]), (s.vval, qkv[t, Hq + Hkv:].to(ref.F64))):
                if quant == BF:
                    val[at] = y.float().bfloat16().to(ref.F64)
                else:
                    q8, e = in_8_bits(y)
                    val[at] = torch.ldexp(q8, e[:, None].int() - 127)
        close(s, out)


def test_streams_at_once():
    """Four layers' calls on four streams, each with its own workspace and cache."""
    made = []
    for i in range(4):
        s = Seqs([700 + 100 * i, 60], Hq=8, Hkv=2, seed=i, quant=(BF, F8)[i % 2])
        p = Seqs([300 + i, 60], [100 + i, 60], Hq=8, Hkv=2, seed=i, quant=(F8, BF)[i % 2])
        made.append((s, p, s.cuda(), p.cuda(), ep.new_attn_workspace(2, 8, 2, 128), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = []
        for s, p, (c1, q1, x1), (c2, q2, x2), ws, st in made:
            outs.append((ep.ep_attn_decode(c1, q1, x1, workspace=ws, stream=st),
                         ep.ep_attn_prefill(c2, q2, x2, stream=st)))
    torch.cuda.synchronize()
    for (s, p, *_), (a, b) in zip(made, outs):
        close(s, a)
        close(p, b)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("quant", [BF, F8])
def test_queries_that_are_not_finite(quant, decode):
    """A query with a NaN or an infinity is NaN, and only that one."""
    def make():
        return Seqs([300, 77], None if decode else [200, 77], Hq=8, Hkv=2, quant=quant)
    s, clean = make(), make()
    s.q[0, 1, 5], s.q[1, 3, 0], s.q[1, 7, 100] = float("nan"), float("inf"), float("-inf")
    out, _ = run(s, decode)
    want, noise, _, _ = clean.attention()
    hit = torch.zeros((s.T, s.Hq), dtype=torch.bool)
    hit[0, 1] = hit[1, 3] = hit[1, 7] = True
    assert torch.isnan(out.cpu()[hit]).all()
    ref.close_bf16(out.cpu()[~hit], want[~hit], noise[~hit])


def test_two_threads():
    """Calls from two host threads, each with handles, a stream and a workspace of its own."""
    import threading
    made, wrong = [], []
    for i in range(2):
        s = Seqs([400 + i, 60], Hq=8, Hkv=2, seed=i, quant=(BF, F8)[i])
        p = Seqs([300 + i, 60], [100 + i, 60], Hq=8, Hkv=2, seed=i, quant=(F8, BF)[i])
        made.append((s, p, s.cuda(), p.cuda(), ep.new_attn_workspace(2, 8, 2, 128), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(s, p, a, b, ws, stream):
        try:
            for _ in range(20):
                x = ep.ep_attn_decode(*a, workspace=ws, stream=stream)
                y = ep.ep_attn_prefill(*b, stream=stream)
            stream.synchronize()
            close(s, x)
            close(p, y)
        except BaseException as e:  # noqa: BLE001 - a thread's failure is the test's
            wrong.append(e)

    threads = [threading.Thread(target=work, args=m) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_attention_beside_the_experts():
    """One layer: norm, append, attention, norm, the few-token experts; programmatic launches all."""
    T, H, Hq, Hkv, D = 3, 512, 4, 2, 128
    s = Seqs([40, 9, 130], Hq=Hq, Hkv=Hkv, D=D)
    cache, seqs, _ = s.cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    x, wn = rand(T, H).bfloat16(), torch.ones(H, device="cuda").bfloat16()
    wqkv, wo = (rand(H, (Hq + 2 * Hkv) * D) / 20).bfloat16(), (rand(Hq * D, H) / 20).bfloat16()
    cs = angles(200, D).cuda()

    def layer():
        n, _, _, _ = ep.ep_rmsnorm(x, wn)
        qkv = (n @ wqkv).view(T, Hq + 2 * Hkv, D)
        q = ep.ep_kv_append(cache, seqs, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cos_sin=cs,
                            q=qkv[:, :Hq])
        a = ep.ep_attn_decode(cache, seqs, q)
        y = a.view(T, Hq * D) @ wo
        n2, _, _, res = ep.ep_rmsnorm(y, wn, residual=x)
        return q, a, n2, res

    q, a, n2, res = layer()
    for _ in range(5):
        again = layer()
        assert all(torch.equal(u, v) for u, v in zip(again, (q, a, n2, res)))
    seqs.check_status()
    s.q = q.cpu()
    s.kval, s.vval = cache.k.cpu().to(ref.F64), cache.v.cpu().to(ref.F64)
    close(s, a)
