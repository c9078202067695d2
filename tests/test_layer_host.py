"""Host-side argument rules of ep_rmsnorm, ep_expert_gemm, ep_expert_swiglu and
ep_moe_decode: every refusal returns before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from tests import layer_ref as ref
from tests.test_abi_host import _layout, lib  # noqa: F401

OK, INVALID, CAPACITY, UNSUPPORTED = 0, 1, 2, 5
P = ctypes.c_void_p
A = P(4096)  # an aligned address that is never read


def _filled(**kw):
    c = _layout(**kw)
    c.dst_row = c.expert_count = c.expert_offset = c.status = 256
    return c


def test_rmsnorm_arguments(lib):  # noqa: F811
    def call(x=A, res=None, w=A, eps=1e-6, T=4, H=256, quant=0, res_out=None, out=A, rows=None,
             scales=None):
        return lib.ep_rmsnorm(x, res, w, eps, T, H, quant, res_out, out, rows, scales, None)

    assert call(T=0) == OK
    for bad in (dict(T=-1), dict(H=0), dict(H=132), dict(H=32776), dict(quant=9), dict(quant=-1),
                dict(x=None), dict(w=None), dict(out=None), dict(x=P(4104)), dict(w=P(4098)),
                dict(res=P(4100)), dict(res_out=P(4100)), dict(out=P(4100)), dict(eps=-1e-6),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=A), dict(scales=A),
                dict(quant=1), dict(quant=1, rows=A), dict(quant=1, scales=A),
                dict(quant=1, rows=P(4100), scales=A), dict(quant=1, rows=A, scales=P(4098)),
                dict(quant=1, H=264, rows=A, scales=A)):
        assert call(**bad) == INVALID, bad


@pytest.mark.parametrize("gated", [False, True])
def test_expert_arguments(lib, gated):  # noqa: F811
    def call(L=None, rows=A, rs=A, H=256, quant=1, w=A, ws=A, n=256, out_quant=1, out=A, os=A):
        L = ctypes.byref(_filled() if L is None else L)
        if gated:
            return lib.ep_expert_swiglu(L, rows, rs, H, quant, w, ws, n, out_quant, out, os, None)
        return lib.ep_expert_gemm(L, rows, rs, H, quant, w, ws, n, out, None)

    assert call(L=_filled(num_tokens=0)) == OK
    bad = [dict(L=_layout()), dict(L=_filled(num_topk=33)), dict(rows=None), dict(rs=None),
           dict(w=None), dict(ws=None), dict(out=None), dict(rows=P(4104)), dict(rs=P(4098)),
           dict(w=P(4104)), dict(ws=P(4098)), dict(out=P(4104)), dict(H=0), dict(H=200),
           dict(H=32896), dict(n=0), dict(n=-8), dict(n=12), dict(n=1 << 20), dict(quant=7)]
    if gated:
        bad += [dict(n=192), dict(os=None), dict(os=P(4098)), dict(out_quant=0),
                dict(out_quant=8)]
    for kw in bad:
        assert call(**kw) == INVALID, kw
    assert call(quant=0) == UNSUPPORTED and call(quant=3) == UNSUPPORTED
    if gated:
        assert call(out_quant=3) == UNSUPPORTED
    assert call(L=_filled(max_tokens=8)) == CAPACITY


@pytest.mark.parametrize("gated", [False, True])
def test_a_made_up_masked_layout_needs_only_what_is_read(lib, gated):  # noqa: F811
    """kind, num_experts, capacity, expert_count and status; all else is zero.  No
    call gets as far as a launch: an mxfp8 call that is not refused for its layout
    answers EP_ERR_UNSUPPORTED, and one without rows EP_ERR_INVALID_ARG, so the
    layout's num_tokens = 0 did not end it."""
    from combine_expert_histogram_gb300.binding import _Layout

    def call(rows=A, quant=1, **kw):
        c = _Layout(num_experts=8, kind=1, capacity=4, expert_count=256, status=256)
        for k, v in kw.items():
            setattr(c, k, v)
        if gated:
            return lib.ep_expert_swiglu(ctypes.byref(c), rows, A, 256, quant, A, A, 256, 1, A, A,
                                        None)
        return lib.ep_expert_gemm(ctypes.byref(c), rows, A, 256, quant, A, A, 256, A, None)

    assert call(quant=3) == UNSUPPORTED
    for other in (dict(num_tokens=-3), dict(num_topk=99), dict(num_ranks=7), dict(align=5),
                  dict(num_tokens=9, max_tokens=8), dict(dst_row=3), dict(expert_offset=3),
                  dict(row_src=1), dict(rank_rows=1)):
        assert call(quant=3, **other) == UNSUPPORTED, other
    assert call(rows=None) == INVALID and call(rows=P(4104)) == INVALID
    for bad in (dict(num_experts=0), dict(num_experts=1025), dict(capacity=0), dict(capacity=-4),
                dict(expert_count=None), dict(expert_count=258), dict(status=None),
                dict(status=257), dict(capacity=1 << 30), dict(kind=2)):
        assert call(quant=3, **bad) == INVALID, bad


def test_moe_decode_arguments(lib):  # noqa: F811
    big = 1 << 40

    def call(x=A, xs=None, quant=0, idx=A, w=A, T=4, K=2, E=8, H=256, I=128, w13=A, s13=A, w2=A,
             s2=A, out=A, status=A, ws=A, n=big):
        return lib.ep_moe_decode(x, xs, quant, idx, w, T, K, E, H, I, w13, s13, w2, s2, out,
                                 status, ws, n, None)

    assert call(T=0) == OK
    for p in ("x", "idx", "w", "w13", "s13", "w2", "s2", "out", "status", "ws"):
        assert call(**{p: None}) == INVALID, p
        assert call(**{p: P(4097)}) == INVALID, p
    for bad in (dict(T=-1), dict(K=0), dict(K=33), dict(E=0), dict(E=1025), dict(H=0),
                dict(H=200), dict(I=64), dict(H=16512), dict(I=16512), dict(quant=9),
                dict(xs=A), dict(quant=1), dict(quant=2), dict(quant=1, xs=P(4098)),
                dict(n=lib.ep_moe_decode_workspace_bytes(4, 2, 8, 256, 128) - 1)):
        assert call(**bad) == INVALID, bad
    assert call(quant=3, xs=A) == UNSUPPORTED and call(quant=4, xs=A) == UNSUPPORTED
    assert call(T=513) == CAPACITY
    assert lib.ep_moe_decode_workspace_bytes(513, 2, 8, 256, 128) == 0
    assert lib.ep_moe_decode_workspace_bytes(512, 2, 8, 256, 128) > 0


@pytest.mark.parametrize("K,E,H,I", [(8, 256, 7168, 2048), (8, 128, 2048, 768), (2, 8, 4096, 14336),
                                     (1, 1, 128, 128), (4, 60, 2048, 1408)])
def test_moe_decode_workspace_serves_fewer_tokens(lib, K, E, H, I):  # noqa: F811
    """Few entries are cut into more parts, so the exact need is not monotone; the
    size that is handed out is."""
    sizes = [lib.ep_moe_decode_workspace_bytes(T, K, E, H, I) for T in range(1, 1024 // K + 1)]
    assert all(a > 0 for a in sizes) and sizes == sorted(sizes)
    # the partial sums of every entry: 2I and H of fp32, in up to four parts
    for T, n in enumerate(sizes, 1):
        assert T * K * 4 * (2 * I + H) <= n <= T * K * 16 * (2 * I + H)


def test_python_calls_refuse_cpu_tensors(lib):  # noqa: F811
    from combine_expert_histogram_gb300 import binding as ep
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm(x, x[0])
    with pytest.raises(ValueError):
        ep.ep_moe_decode(x, i, i.float(), x, x, x, x)


def _cpu_slab(E=3, cap=4):
    from combine_expert_histogram_gb300 import binding as ep
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    return ep.Layout(6, 2, E, 1, "masked", 1, cap, 0, dst_row=i32(12), row_src=None,
                     expert_count=i32(E), expert_offset=i32(E + 1), rank_rows=None,
                     status=i32(1))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("which", ["rows", "scales"])
def test_a_slab_cut_out_of_a_larger_one_is_refused(lib, gated, which):  # noqa: F811
    """[E, capacity, ...] views of a larger slab are no contiguous rows: a copy of
    them would be freed before the launch."""
    from combine_expert_histogram_gb300 import binding as ep
    E, cap, K = 3, 4, 256
    rows = torch.zeros((E, cap + 2, K), dtype=torch.uint8)
    sc = torch.zeros((E, cap + 2, K // 128))
    w, ws = torch.zeros((E, 256, K), dtype=torch.uint8), torch.zeros((E, 2, K // 128))
    if which == "rows":
        rows, sc = rows[:, :cap], sc[:, :cap].contiguous()
    else:
        rows, sc = rows[:, :cap].contiguous(), sc[:, :cap]
    with pytest.raises(ValueError, match="contiguous"):
        (ep.ep_expert_swiglu if gated else ep.ep_expert_gemm)(_cpu_slab(E, cap), rows, sc, w, ws)


def test_the_rows_of_a_slab_share_its_memory():
    from combine_expert_histogram_gb300 import binding as ep
    for shape in ((3, 4, 256), (1, 1, 128), (2, 0, 128)):
        t = torch.zeros(shape)
        r = ep._slab_rows(t)
        assert r.shape == (shape[0] * shape[1], shape[2]) and r.data_ptr() == t.data_ptr()


def test_the_layers_own_workspace_is_sized_on_its_device(lib, monkeypatch):  # noqa: F811
    """Tensors on device 3 while another one is current (a stand-in for both: the
    argument checks pass, the call is recorded): the size is asked for with device
    3 current, as new_moe_workspace does."""
    import contextlib
    from combine_expert_histogram_gb300 import binding as ep
    current, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        old, current[0] = current[0], d if isinstance(d, int) else d.index
        yield
        current[0] = old

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(ep, "_rows_of", lambda t, name, dims=2: 3)
    monkeypatch.setattr(ep, "_want", lambda *a: 256)
    monkeypatch.setattr(ep, "_empty", lambda shape, dtype, dev, stream: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(ep, "_on", lambda stream, dev: 0)
    monkeypatch.setattr(ep, "_call", lambda *a: asked.append("call"))
    monkeypatch.setattr(ep, "ep_moe_decode_workspace_bytes",
                        lambda *a: asked.append((current[0], a)) or 64)
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    idx = torch.zeros((2, 1), dtype=torch.int32)
    ep.ep_moe_decode(torch.zeros((2, 128), dtype=torch.bfloat16), idx, idx.float(),
                     u8(4, 256, 128), torch.zeros(4, 2, 1), u8(4, 128, 128), torch.zeros(4, 1, 1))
    assert asked == [(3, (2, 1, 4, 128, 128)), "call"] and current == [0]


def test_some_quotients_are_moved_by_a_reciprocal():
    """tie_groups has what it promises: values that the quotient and the product by
    the reciprocal quantise differently, so that a kernel with the other rule fails."""
    v = ref.tie_groups(128, torch.Generator().manual_seed(1))
    assert torch.equal(v.bfloat16().float(), v)
    assert torch.equal(v.abs().amax(1), torch.arange(128.0, 256.0))
    s = v[:, :1].abs() / torch.full((128, 1), 448.0)
    inv = (1 / s.double()).float()
    moved = ref.e4m3((v / s).double()) != ref.e4m3((v * inv).double())
    assert moved.sum() >= 60 and moved.any(1).sum() >= 7
    assert torch.equal(ref.quantise_bf16(v)[0], ref.e4m3((v / s).double()))


def test_the_64_bit_e4m3_agrees_with_torch():
    """The test's own E4M3 decoding and rounding against torch's cast."""
    b = torch.arange(256, dtype=torch.uint8)
    v = b.view(torch.float8_e4m3fn).double()
    got = ref.decode(b)
    assert torch.equal(got.isnan(), v.isnan())
    assert torch.equal(got[~v.isnan()], v[~v.isnan()])
    x = torch.cat([torch.randn(20000) * 60, torch.randn(2000) * 1e-3, torch.tensor([0.0, 448.0])])
    x = x.clamp(-448, 448)
    assert torch.equal(ref.e4m3(x.double()), x.to(torch.float8_e4m3fn).double())
    mids = (v[:126] + v[1:127]) / 2  # ties go to the even mantissa
    assert torch.equal(ref.e4m3(mids), mids.float().to(torch.float8_e4m3fn).double())
