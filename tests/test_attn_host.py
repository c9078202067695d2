"""Host-side argument rules of ep_kv_append, ep_attn_decode and ep_attn_prefill: every refusal
returns before any CUDA call (no GPU needed); and the tests' own reference."""
import ctypes

import pytest
import torch

from tests import attn_ref, layer_ref as ref
from tests.test_abi_host import lib  # noqa: F401

OK, INVALID, UNSUPPORTED = 0, 1, 5
P = ctypes.c_void_p
A = P(4096)  # an aligned address that is never read


def cache(**kw):
    from combine_expert_histogram_gb300.binding import _KvCache
    d = dict(num_pages=9, page_size=16, num_kv_heads=2, head_dim=128, quant=0,
             page_stride=16 * 2 * 128, row_stride=128, head_stride=16 * 128, k=4096, v=8192)
    if kw.get("quant") == 2:
        d.update(k_scales=4096, v_scales=4096)
    d.update(kw)
    return _KvCache(**d)


def seqs(**kw):
    from combine_expert_histogram_gb300.binding import _KvSeqs
    d = dict(num_seqs=3, num_tokens=3, max_pages=4, block_table=256, kv_len=256, q_start=None,
             status=256)
    d.update(kw)
    return _KvSeqs(**d)


BAD_CACHE = (dict(num_pages=0), dict(num_pages=-1), dict(page_size=0), dict(page_size=12),
             dict(page_size=8192), dict(num_kv_heads=0), dict(num_kv_heads=1025), dict(head_dim=0),
             dict(quant=-1), dict(quant=9), dict(page_stride=0), dict(page_stride=-4096),
             dict(row_stride=100), dict(head_stride=1 << 40), dict(k=None), dict(v=None),
             dict(k=4104), dict(v=4104), dict(k_scales=4096), dict(v_scales=4096),
             dict(quant=2, k_scales=None), dict(quant=2, v_scales=None),
             dict(quant=2, k_scales=4100), dict(quant=2, v_scales=4100), dict(quant=2, row_stride=136))
BAD_SEQS = (dict(num_seqs=-1), dict(num_tokens=-1), dict(num_tokens=4), dict(max_pages=0),
            dict(max_pages=1 << 30), dict(block_table=None), dict(kv_len=None), dict(status=None),
            dict(block_table=258), dict(kv_len=258), dict(status=258), dict(q_start=258))
ODD_CACHE = (dict(head_dim=96), dict(head_dim=256), dict(quant=1), dict(quant=3), dict(quant=4))


def _entries(lib):  # noqa: F811
    def append(c=None, s=None, q=A, qs=512, Hq=4, k=A, ks=256, v=A, vs=256, cs=A, R=64, n=99,
               inter=0, qo=A, qos=512):
        return lib.ep_kv_append(ctypes.byref(c or cache()), ctypes.byref(s or seqs()), q, qs, Hq, k,
                                ks, v, vs, cs, R, n, inter, qo, qos, None)

    def decode(c=None, s=None, q=A, qs=512, Hq=4, scale=0.1, window=0, sinks=0, out=A, lse=None,
               ws=A, n=1 << 30):
        return lib.ep_attn_decode(ctypes.byref(c or cache()), ctypes.byref(s or seqs()), q, qs, Hq,
                                  scale, window, sinks, out, lse, ws, n, None)

    def prefill(c=None, s=None, q=A, qs=512, Hq=4, scale=0.1, window=0, sinks=0, out=A, lse=None,
                ws=None, n=0):
        return lib.ep_attn_prefill(ctypes.byref(c or cache()), ctypes.byref(s or seqs()), q, qs, Hq,
                                   scale, window, sinks, out, lse, ws, n, None)

    return append, decode, prefill


@pytest.mark.parametrize("which", range(3))
def test_cache_and_sequences(lib, which):  # noqa: F811
    call = _entries(lib)[which]
    for kw in BAD_CACHE:
        assert call(c=cache(**kw)) == INVALID, kw
    for kw in ODD_CACHE:
        assert call(c=cache(**kw)) == UNSUPPORTED, kw
    for kw in BAD_SEQS:
        assert call(s=seqs(**kw)) == INVALID, kw
    assert call(s=seqs(num_seqs=0, num_tokens=0)) == OK
    assert call(s=seqs(num_seqs=0, num_tokens=0, block_table=None, kv_len=None)) == OK
    if which != 1:
        assert call(s=seqs(num_seqs=0, num_tokens=5, q_start=256)) == OK
        assert call(s=seqs(num_seqs=5, num_tokens=0, q_start=256)) == OK
    fn = (lib.ep_kv_append, lib.ep_attn_decode, lib.ep_attn_prefill)[which]
    rest = [0 if t is not P else None for t in fn.argtypes[2:]]
    assert fn(None, ctypes.byref(seqs()), *rest) == INVALID
    assert fn(ctypes.byref(cache()), None, *rest) == INVALID


def test_append_arguments(lib):  # noqa: F811
    call = _entries(lib)[0]
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(q=P(4104)), dict(qo=P(4104)),
               dict(k=P(4104)), dict(v=P(4104)), dict(qs=511), dict(qs=504), dict(ks=255), dict(vs=248),
               dict(ks=-256), dict(qos=516), dict(Hq=-1), dict(Hq=1025), dict(Hq=0), dict(R=-16),
               dict(R=8), dict(R=144), dict(R=0), dict(cs=None), dict(cs=P(4104)), dict(n=-1),
               dict(vs=1 << 40)):
        assert call(**kw) == INVALID, kw


@pytest.mark.parametrize("which", [1, 2])
def test_attention_arguments(lib, which):  # noqa: F811
    call = _entries(lib)[which]
    for kw in (dict(q=None), dict(out=None), dict(q=P(4104)), dict(out=P(4104)), dict(lse=P(4098)),
               dict(qs=504), dict(qs=514), dict(Hq=0), dict(Hq=3), dict(Hq=1026), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
               dict(window=8, sinks=-1)):
        assert call(**kw) == INVALID, kw
    more = ((dict(ws=None), dict(ws=P(4104)), dict(n=8), dict(s=seqs(q_start=256))) if which == 1
            else (dict(ws=P(4104), n=1 << 30), dict(ws=A, n=8)))
    for kw in more:
        assert call(**kw) == INVALID, kw


def test_workspace_sizes(lib):  # noqa: F811
    size = lib.ep_attn_decode_workspace_bytes
    assert size(-1, 4, 2, 128) == size(1, 3, 2, 128) == size(1, 4, 2, 96) == size(1, 0, 1, 64) == 0
    assert size(1, 1025, 1, 64) == 0
    for D in (64, 128):
        for heads in ((1, 1), (4, 2), (32, 4), (64, 1), (1024, 1024)):
            sizes = [size(B, *heads, D) for B in (0, 1, 2, 7, 64, 1000)]
            assert sizes == sorted(sizes) and 0 < sizes[0]


def test_prefill_workspace_sizes(lib):  # noqa: F811
    size = lib.ep_attn_prefill_workspace_bytes
    assert size(-1, 1, 4, 2, 128) == size(1, -1, 4, 2, 128) == size(1, 1, 3, 2, 128) == 0
    assert size(1, 1, 4, 2, 96) == size(1 << 28, 1, 64, 2, 128) == 0
    assert size(1, 1, 4, 2, 128) > size(1, 1, 4, 2, 64) > 0
    assert len({size(T, B, 32, 8, 128) for T in (0, 1, 700, 5000) for B in (0, 1, 40)}) == 1


def test_status_name(lib):  # noqa: F811
    assert lib.ep_status_str(7).startswith(b"EP_ERR_BAD_PAGE")


def test_handles_refuse_cpu_tensors():
    from combine_expert_histogram_gb300 import binding as ep
    x = torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ep.KvCache(x, x)
    i = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        ep.new_kv_seqs(i, i[:, 0].contiguous())


def test_the_reference_itself():
    """Attention by hand for three keys, a rotation by a right angle, 8-bit rows by powers of two."""
    s = attn_ref.Seqs([3], Hq=1, Hkv=1, D=64, page=8)
    k, v = s.rows(0, 0)
    q = s.q[0, 0].to(ref.F64)
    p = torch.exp(k @ q / 8)
    out, noise, lse, _ = s.attention()
    assert torch.allclose(out[0, 0], (p[:, None] * v).sum(0) / p.sum(), atol=1e-12)
    assert abs(float(lse[0, 0] - p.sum().log())) < 1e-12 and float(noise.max()) < 0.05
    out, _, _, _ = s.attention(window=1, sinks=1)
    assert torch.allclose(out[0, 0], (p[0] * v[0] + p[2] * v[2]) / (p[0] + p[2]), atol=1e-12)
    x = torch.arange(1.0, 65.0).to(ref.F64).reshape(1, 1, 64)
    zero, one = torch.zeros(1, 8), torch.ones(1, 8)
    y = attn_ref.rotate(x, zero, one, False)
    assert y[0, 0, :8].tolist() == [-float(i) for i in range(9, 17)]
    assert y[0, 0, 8:16].tolist() == [float(i) for i in range(1, 9)] and y[0, 0, 16] == 17
    y = attn_ref.rotate(x, zero, one, True)
    assert y[0, 0, :4].tolist() == [-2, 1, -4, 3]
    q8, e = attn_ref.in_8_bits(torch.tensor([[448.0, 1.0], [449.0, 2.0], [0.0, 0.0]]).to(ref.F64))
    assert e.tolist()[:2] == [127, 128] and q8[0].tolist() == [448, 1] and q8[1].tolist() == [224, 1]
