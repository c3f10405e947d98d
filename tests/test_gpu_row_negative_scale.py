"""run_shared_prefix with a scale below zero: tiles of 128 rows, of more, and a batch with both."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention
from row_attn_ref import check, make, poison
from row_attn_ref import reference as loose
from row_terms_ref import make_terms, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own,prefix,hq,hkv,d,bs,dtype", [
    ([5] * 9 + [130], 700, 16, 2, 128, 16, torch.bfloat16),
    ([40] * 17, 640, 16, 2, 64, 16, torch.float16),
    ([33, 200] * 20, 1024, 8, 1, 128, 32, torch.bfloat16),
])
def test_negative_scale(own, prefix, hq, hkv, d, bs, dtype):
    n, lens = len(own), [prefix + x for x in own]
    cu, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [prefix]))
    args = make(lens, hq, hkv, d, bs, dtype, [(0, n, prefix)], seed=7)
    poison(args[1], args[2], args[3], args[4])
    terms = make_terms(lens, hq, hkv, d, bs, dtype, [(0, n, prefix)], seed=8, scale=-1.0, device="cuda")
    with PagedDecodeAttention(hq, hkv, d, bs, dtype, max_batch=n, max_blocks_per_seq=args[3].shape[1], max_splits=1) as a:
        for cap in (0.0, 3.0):
            check(a.run_shared_prefix(*args, cu, pre, -0.2, cap), *loose(*args, -0.2, cap))
            check(a.run_shared_prefix(*terms, cu, pre, -1.0, cap), *reference(*terms, -1.0, cap))
