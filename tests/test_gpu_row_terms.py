"""run_shared_prefix and run(softcap, alibi_slopes, window): the weights are the sum of two 16-bit
terms in every tile, whoever else is in the batch."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention
from row_attn_ref import check
from row_terms_ref import OWN, SHARED, make_terms, reference

pytestmark = pytest.mark.gpu


def handle(q, k, table):
    nb, bs, hkv, d = k.shape
    return PagedDecodeAttention(q.shape[1], hkv, d, bs, q.dtype, max_batch=len(q),
                                max_blocks_per_seq=table.shape[1], max_splits=1)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cap,alibi", [(0.0, False), (2.0, False), (0.0, True)])
@pytest.mark.parametrize("own,prefix,hq,hkv,d,bs,dtype", SHARED)
def test_shared_tiles(own, prefix, hq, hkv, d, bs, dtype, cap, alibi):
    n = len(own)
    args = make_terms([prefix + x for x in own], hq, hkv, d, bs, dtype, [(0, n, prefix)], seed=5, device="cuda")
    slopes = torch.linspace(1e-4, 2e-3, hq).cuda() if alibi else None
    with handle(args[0], args[1], args[3]) as a:
        out = a.run_shared_prefix(*args, ints(0, n), ints(prefix), 1.0, cap, slopes)
        assert a.check_device_error() == (0, 0)
    check(out, *reference(*args, 1.0, cap, slopes))


@pytest.mark.parametrize("lens,hq,hkv,d,bs,dtype,cap,window", OWN)
def test_own_tiles(lens, hq, hkv, d, bs, dtype, cap, window):
    args = make_terms(lens, hq, hkv, d, bs, dtype, seed=6, device="cuda")
    with handle(args[0], args[1], args[3]) as a:
        out = a.run(*args, 1.0, softcap=cap, window=window)
        assert a.check_device_error() == (0, 0)
    check(out, *reference(*args, 1.0, cap, None, window))
