"""An infinity in a row of V that is attended to: the result of its dim is not finite, and nothing
else changes."""
import math

import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention
from row_attn_ref import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d,seqs", [(8, 2, 128, 3), (16, 2, 64, 40), (16, 1, 128, 9)])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_infinity_stays_in_its_dim(dtype, hq, hkv, d, seqs, value):
    lens = [400 + 3 * i for i in range(seqs)]
    q, k, v, table, ln = make(lens, hq, hkv, d, 16, dtype, [(0, seqs, 384)], seed=9)
    cu, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, seqs], [384]))
    bad = v.clone()
    bad[table[1, 24].long(), 2, 0, 5] = value  # a token of the second sequence's own part, kv head 0
    with PagedDecodeAttention(hq, hkv, d, 16, dtype, max_batch=seqs, max_blocks_per_seq=table.shape[1], max_splits=1) as a:
        for call in (lambda x: a.run_shared_prefix(q, k, x, table, ln, cu, pre, 0.1),
                     lambda x: a.run(q, k, x, table, ln, 0.1, softcap=9.0),
                     lambda x: a.run(q, k, x, table, ln, 0.1, window=300)):
            want, got = call(v), call(bad)
            hit = torch.zeros_like(want, dtype=torch.bool)
            hit[1, :hq // hkv, 5] = True
            assert not torch.isfinite(got[hit]).any()
            assert torch.equal(got[~hit], want[~hit])
        # in the shared part it reaches every sequence of the group
        bad = v.clone()
        bad[table[0, 3].long(), 7, hkv - 1, 0] = value
        want, got = (a.run_shared_prefix(q, k, x, table, ln, cu, pre, 0.1) for x in (v, bad))
        hit = torch.zeros_like(want, dtype=torch.bool)
        hit[:, hq - hq // hkv:, 0] = True
        assert not torch.isfinite(got[hit]).any()
        assert torch.equal(got[~hit], want[~hit])
        assert a.check_device_error() == (0, 0)
