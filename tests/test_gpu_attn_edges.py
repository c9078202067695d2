"""The paged cache and its attention where their numbers and lists end: short pieces of many
sequences, addresses, tables and values at the edges of what include/ep.h allows."""
import pytest
import torch

from combine_expert_histogram_gb300 import binding as ep
from tests.attn_ref import Seqs, close

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
