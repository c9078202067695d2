"""The paged cache and its attention where their numbers and lists end: short pieces of many
sequences, addresses, tables and values at the edges of what include/ep.h allows."""
import ctypes
import math

import pytest
import torch

from combine_expert_histogram_gb300 import binding as ep
from tests import layer_ref as ref
from tests.attn_ref import Seqs, close, in_8_bits

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF, F8 = "none", "fp8_ue8m0"


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,n,window", [(48, 4, 0), (128, 4, 0), (128, 1, 64), (48, 1, 0)])
def test_prefill_of_many_short_sequences(B, n, window, D, quant):
    """Row blocks of one and of few key tiles one after another in an SM's run, whose halves meet
    the ring at every place; the same bits each time, with the cache in L2 or not."""
    g = torch.Generator().manual_seed(B + n)
    lens = torch.randint(50, 401, (B,), generator=g).tolist()
    s = Seqs(lens, [n] * B, Hq=8, Hkv=8, D=D, quant=quant, page=16)
    cache, seqs, q = s.cuda()
    out = ep.ep_attn_prefill(cache, seqs, q, window=window)
    seqs.check_status()
    close(s, out, window=window, device="cuda")
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(8):
        if i % 2:
            big.fill_(i)
        assert torch.equal(ep.ep_attn_prefill(cache, seqs, q, window=window), out)
    seqs.check_status()


def offset(t, nbytes):
    """A contiguous copy of t that begins nbytes behind an aligned address."""
    raw = torch.empty(t.numel() * t.element_size() + nbytes, dtype=torch.uint8, device="cuda")
    part = raw[nbytes:].view(t.dtype).view(t.shape)
    part.copy_(t)
    assert part.data_ptr() % 512 == nbytes
    return part


@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
def test_addresses_of_sixteen_bytes(D, quant):
    """Rows, results and scratch that begin at a multiple of 16 bytes and of no more: the same
    bits; of 8 bytes: refused."""
    s = Seqs([700, 300, 9], [300, 5, 9], Hq=8, Hkv=2, D=D, quant=quant, page=24)
    cache, seqs, q = s.cuda()
    want = ep.ep_attn_prefill(cache, seqs, q)
    n = ep.ep_attn_prefill_workspace_bytes(s.T, 3, 8, 2, D)
    for at in (16, 48):
        out, lse = offset(torch.zeros_like(q), at), offset(torch.zeros((s.T, 8), device="cuda"), 4)
        scratch = offset(torch.zeros(n, dtype=torch.uint8, device="cuda"), at)
        ep.ep_attn_prefill(cache, seqs, offset(q, at), out=out, lse=lse, scratch=scratch)
        assert torch.equal(out, want)
    close(s, out, lse)
    one = Seqs([700, 300, 9], Hq=8, Hkv=2, D=D, quant=quant, page=24)
    c1, s1, q1 = one.cuda()
    ws = ep.AttnWorkspace(offset(torch.zeros(ep.ep_attn_decode_workspace_bytes(3, 8, 2, D), dtype=torch.uint8,
                                             device="cuda"), 16))
    got = ep.ep_attn_decode(c1, s1, offset(q1, 16), workspace=ws, out=offset(torch.zeros_like(q1), 16))
    assert torch.equal(got, ep.ep_attn_decode(c1, s1, q1))
    k = torch.randn((s.T, 2, D), generator=s.g).bfloat16().cuda()
    tables = torch.cat([torch.ones((700, D // 2)), torch.zeros((700, D // 2))], 1).cuda()
    rot = ep.ep_kv_append(cache, seqs, offset(k, 16), offset(k, 48), cos_sin=offset(tables, 16), q=offset(q, 16),
                          q_out=offset(torch.zeros_like(q), 48))
    assert torch.equal(rot, q)
    seqs.check_status()
    for kw in (dict(out=offset(torch.zeros_like(q), 8)),
               dict(scratch=offset(torch.zeros(n, dtype=torch.uint8, device="cuda"), 8))):
        with pytest.raises(ep.EPError):
            ep.ep_attn_prefill(cache, seqs, q, **kw)


@pytest.mark.parametrize("quant", [BF, F8])
def test_append_past_the_block_table(quant):
    """Tokens past a block table are skipped, whatever the length says; those before its end are
    stored where they belong, and what the cache held stays."""
    for length, n in ((41, 4), (42, 4), (43, 4), (44, 4), (48, 4), (1000, 4), ((1 << 31) - 1, 4), (40, 4), (45, 40)):
        s = Seqs([40, 20], [n, 2], Hq=2, Hkv=2, D=64, page=8, quant=quant, extra_cols=0)
        cache, seqs, _ = s.cuda()
        seqs.kv_len[0] = length
        k = torch.randn((s.T, 2, 64), generator=s.g).bfloat16()
        q = torch.randn((s.T, 2, 64), generator=s.g).bfloat16().cuda()
        nan = torch.full((s.T, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        cos, sin = torch.ones((2000, 32)), torch.zeros((2000, 32))  # no turn: rows as they are
        kept = [t.clone() for t in (cache.k, cache.v)]
        scales = [] if quant == BF else [t.clone() for t in (cache.k_scales, cache.v_scales)]
        out = ep.ep_kv_append(cache, seqs, k.cuda(), k.cuda(), cos_sin=torch.cat([cos, sin], 1).cuda(), q=q, q_out=nan)
        torch.cuda.synchronize()
        if length > 40:
            with pytest.raises(ep.EPError) as e:
                seqs.check_status()
            assert e.value.code == ep.EP_ERR_BAD_PAGE
        else:
            seqs.check_status()
        stored = [(t, 0, length - n + t) for t in range(n) if 0 <= length - n + t < 40]
        stored += [(n, 1, 18), (n + 1, 1, 19)]
        at = [x for x, _, _ in stored]
        page = torch.tensor([int(s.table[b, i // 8]) for _, b, i in stored])
        row = torch.tensor([i % 8 for _, _, i in stored])
        rest = [t for t in range(s.T) if t not in at]
        assert torch.equal(out[at], q[at]) and torch.isnan(out[rest]).all()
        rows, e8 = (k[at], None) if quant == BF else in_8_bits(k[at].to(ref.F64))
        if quant == F8:
            rows = rows.float().to(torch.float8_e4m3fn).view(torch.uint8)
        bits = torch.int16 if quant == BF else torch.uint8
        for was, now in zip(kept, (cache.k, cache.v)):
            want = was.cpu()
            want[page, row] = rows
            assert torch.equal(now.cpu().view(bits), want.view(bits))
        for was, now in zip(scales, (cache.k_scales, cache.v_scales)):
            want = was.cpu()
            want[page, :, row] = e8
            assert torch.equal(now.cpu(), want)


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("drop", [0.75, 3.0, 4.0])
def test_a_million_equal_logits(drop, decode):
    """The sum of a long row's probabilities: a tile's are added by themselves, then to the row's.  All
    values are 1, so that the result is 1; shared out among blocks, and by one (prompts)."""
    L, page, D = 1 << 20, 128, 64
    k, v = torch.zeros((L // page, 1, page, D)), torch.ones((L // page, 1, page, D))
    k[0, 0, 0, 0] = k[1, 0, 0, 0] = drop  # in a tile of each half
    cache = ep.KvCache(k.bfloat16().cuda().transpose(1, 2), v.bfloat16().cuda().transpose(1, 2))
    table = torch.arange(L // page, dtype=torch.int32)[None].cuda()
    seqs = ep.new_kv_seqs(table, torch.tensor([L], dtype=torch.int32).cuda())
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    out, lse = torch.zeros_like(q), torch.zeros((1, 1), device="cuda")
    want = math.log(2 * math.exp(drop) + L - 2)
    # logits are exact.  Of the sum, relative: an exponential's 2^-22 and four roundings of its
    # argument, one rounding for each of half the tiles' sums, and 64 for a tile's own chain and the joins
    # (single tokens: a chain of 2^20 / 64 at most); the logarithm's 2^-22, four roundings of the result
    rel = 2.0 ** -22 + 4 * ref.U * 2 * drop + ref.U * ((L // 64 if decode else L // 256) + 64)
    off = rel + 2.0 ** -22 + 4 * ref.U * (drop + want)

    def check():
        assert abs(float(lse) - want) <= off, (float(lse), want, off)
        assert ((out.double() - 1).abs() <= ref.BF16 + 2 * ref.BF16).all()  # P's rounding, and the result's

    if decode:
        ep.ep_attn_decode(cache, seqs, q, scale=1.0, out=out, lse=lse)
        return check()
    ep.ep_attn_prefill(cache, seqs, q, scale=1.0, out=out, lse=lse)
    check()
    code = ep.load_library().ep_attn_prefill(ctypes.byref(cache._c), ctypes.byref(seqs._struct(1)), q.data_ptr(), D, 1,
                                             1.0, 0, 0, out.data_ptr(), lse.data_ptr(), None, 0, None)
    assert code == 0
    torch.cuda.synchronize()
    check()


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_values_past_bf16(D):
    """An 8-bit value that bf16 does not hold (the largest bf16, appended, is 2^128) is an infinity in every
    row that sees it, in tiles that all rows see and in others."""
    def make():
        return Seqs([400], [400], Hq=2, Hkv=1, D=D, quant=F8)
    s = make()
    for j in (20, 150, 300):
        p, r = s.table[0, j // s.page].long(), j % s.page
        s.v[p, r, 0], s.vs[p, 0, r] = 0, 247
        s.v[p, r, 0, 5], s.v[p, r, 0, 6] = 0x78, 0xF8  # 256 * 2^120
    big = torch.full((1, 1, D), 3.3895e38).bfloat16()  # what ep_kv_append makes of such a row
    q8, e = in_8_bits(big.to(ref.F64))
    assert int(e) == 247 and float(q8.max()) == 256
    for window, sees in ((0, lambda i: i >= 20), (30, lambda i: any(j <= i < j + 30 for j in (20, 150, 300)))):
        cache, seqs, q = s.cuda()
        out = ep.ep_attn_prefill(cache, seqs, q, window=window).cpu()
        seqs.check_status()
        seen = torch.tensor([sees(i) for i in range(400)])
        assert (out[seen][..., 5] == float("inf")).all() and (out[seen][..., 6] == float("-inf")).all()
        assert torch.isfinite(out[~seen]).all()
        # the others' channels: the row's values there are zeros
        clean = make()
        for j in (20, 150, 300):
            clean.vval[clean.table[0, j // s.page].long(), j % s.page] = 0
        want, noise, _, _ = clean.attention(window=window)
        rest = [d for d in range(D) if d not in (5, 6)]
        ref.close_bf16(out[..., rest], want[..., rest], noise[..., rest])


@pytest.mark.parametrize("Hq", [4, 32])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_infinite_value_that_is_seen(D, Hq):
    """An infinite value channel is infinite in every head that sees it, the others are not."""
    lens = [200, 1, 5000, 40]
    s, clean = (Seqs(lens, Hq=Hq, Hkv=2, D=D) for _ in range(2))
    at = ((0, 150), (1, 0), (2, 77), (2, 4001))
    for b, j in at:
        p, r = s.table[b, j // s.page].long(), j % s.page
        s.v[p, r, 0, 9], s.v[p, r, 0, 30] = float("-inf"), float("inf")
    cache, seqs, q = s.cuda()
    out = ep.ep_attn_decode(cache, seqs, q).cpu()
    G = Hq // 2
    assert (out[:3, :G, 9] == float("-inf")).all() and (out[:3, :G, 30] == float("inf")).all()
    want, noise, _, _ = clean.attention()
    rest = [d for d in range(D) if d not in (9, 30)]
    ref.close_bf16(out[..., rest], want[..., rest], noise[..., rest])
    ref.close_bf16(out[:, G:], want[:, G:], noise[:, G:])
    ref.close_bf16(out[3], want[3], noise[3])


def test_decode_probabilities_keep_sixteen_bits():
    """One key of value 0 and one of value v: the result p v / (1 + p) has no rounding of p to 8 bits
    (2^-16 is what two bf16 leave of it), only the result's own."""
    D, B = 128, 64
    s = Seqs([2] * B, Hq=8, Hkv=2, D=D, page=8)
    p = s.table[:, 0].long()
    s.v[p, 0] = 0
    s.vval = s.v.to(ref.F64)
    cache, seqs, q = s.cuda()
    out = ep.ep_attn_decode(cache, seqs, q).cpu().to(ref.F64)
    want, _, _, _ = s.attention()
    k = s.kval[p, :2]  # [B, 2, Hkv, D]
    mag = torch.einsum("bhgd,bjhd->bhgj", s.q.to(ref.F64).abs().view(B, 2, 4, D), k.abs()).amax(-1).reshape(B, 8, 1)
    # two logits and exponentials, p and the sums
    off = 2 * (2 * (D + 4) * ref.U * D ** -0.5 * mag + 2.0 ** -20) + 2.0 ** -16 + 2.0 ** -20
    half = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -100)))) * ref.BF16
    assert ((out - want).abs() <= half + want.abs() * off).all()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("quant", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
def test_logits_of_minus_infinity(D, quant, decode):
    """A row that sees keys, whose logits are all -infinity, is 0 / 0, not a row without keys."""
    lens = [1, 0, 300, 5000]
    new = None if decode else [1, 0, 2, 1]
    s = Seqs(lens, new, Hq=4, Hkv=1, D=D, quant=quant)
    if quant == BF:
        s.k[..., 3] = s.k[..., 3].abs() + 1
    else:
        s.k[..., 3] = 0x38  # 1
    s.q[..., 3] = 1.0
    s.q[:, 1, 3] = float("-inf")
    cache, seqs, q = s.cuda()
    lse = torch.zeros((s.T, 4), device="cuda")
    out = (ep.ep_attn_decode if decode else ep.ep_attn_prefill)(cache, seqs, q, lse=lse).cpu()
    rows = [t for t in range(s.T) if not (decode and t == 1)]
    assert torch.isnan(out[rows, 1]).all() and torch.isfinite(out[:, [0, 2, 3]]).all()
    assert (lse.cpu()[rows, 1] == float("-inf")).all()
    if decode:
        assert (out[1] == 0).all() and (lse[1] == float("-inf")).all()


@pytest.mark.parametrize("D", [64, 128])
def test_decode_large_logits_of_8_bit_keys(D):
    """Products that fp32 holds, although 2^8 times as large ones would not be: one key takes it all."""
    s = Seqs([50, 900], Hq=4, Hkv=1, D=D, quant=F8)
    s.k[..., 1:] = 0
    s.k[..., 0] = torch.randint(1, 0x70, s.k[..., 0].shape, generator=s.g).to(torch.uint8)
    s.ks[:] = 245  # 2^118
    s.q[:] = 0
    s.q[..., 0] = 0.5
    best = []
    for b, L in enumerate(s.lens):
        j = L // 3
        p, r = s.table[b, j // s.page].long(), j % s.page
        s.k[p, r, 0, 0] = 0x7E  # 448
        best.append(s.vval[p, r, 0])
    cache, seqs, q = s.cuda()
    lse = torch.zeros((2, 4), device="cuda")
    out = ep.ep_attn_decode(cache, seqs, q, lse=lse).cpu()
    for b in range(2):
        assert torch.equal(out[b].float(), best[b].float().expand(4, D))
    want = 448 * 2.0 ** 117 * D ** -0.5
    assert (abs(lse.cpu().double() / want - 1) <= 8 * ref.U).all()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_the_smallest_and_largest_scales(D, decode):
    """Results down to bf16's smallest normal numbers and up to its largest; zeros beside the largest stay
    zeros."""
    for byte in (0, 1, 3, 120, 240, 246, 254):
        s = Seqs([300, 40, 1], None if decode else [3, 1, 1], Hq=12, Hkv=1, D=D, quant=F8)
        s.vs[:] = byte
        s.v[:] = torch.randint(0x38, 0x3C, s.v.shape, generator=s.g).to(torch.uint8)  # 1 to 1.375
        if byte == 254:
            s.v[..., 1::2] = 0
        s.vval = torch.ldexp(ref.decode(s.v), torch.tensor(byte - 127))
        cache, seqs, q = s.cuda()
        out = (ep.ep_attn_decode if decode else ep.ep_attn_prefill)(cache, seqs, q).cpu()
        want, noise, _, _ = s.attention()
        if byte == 254:
            # sums are in fp32 before the division: of 2^127 and more, times probabilities that sum up to
            # more than 2, they are past 2^128.  The one key of the last row has the probability 1.
            assert (out[..., 1::2] == 0).all() and (out[..., ::2] > 0).all()
            out, want, noise = out[-1:], want[-1:], noise[-1:]
        ref.close_bf16(out, want, noise)
