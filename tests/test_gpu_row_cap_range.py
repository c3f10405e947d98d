"""Caps and scales at the ends of fp32's range: served right, or refused."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PDA_EINVAL, PDAError, PagedDecodeAttention
from row_attn_ref import check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def call():
    q, k, v, table, ln = make([300, 170], 8, 2, 128, 16, torch.bfloat16, [(0, 2, 160)], seed=41)
    k[table[0, 2].long()] = 0  # some products are exactly zero
    cu, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2], [160]))
    a = PagedDecodeAttention(8, 2, 128, 16, torch.bfloat16, max_batch=2, max_blocks_per_seq=table.shape[1], max_splits=1)

    def both(scale, cap):
        return (a.run(q, k, v, table, ln, scale, softcap=cap, window=10 ** 6),
                a.run_shared_prefix(q, k, v, table, ln, cu, pre, scale, cap)), (q, k, v, table, ln)
    yield both
    a.close()


@pytest.mark.parametrize("scale,cap", [(0.1, 8.0e36), (4.0, 2.3e38), (0.1, 1e30), (0.1, 1e-37), (0.0, 3e-39),
                                       (0.0, 2.3e38), (1e-30, 50.0), (-0.1, 8.0e36)])
def test_served(call, scale, cap):
    outs, args = call(scale, cap)
    want = reference(*args, scale, cap)
    for out in outs:
        check(out, *want)


@pytest.mark.parametrize("scale,cap", [(0.1, 3.0e38), (0.1, 1.0e38), (0.1, 1.0e37), (1e-8, 1e38), (4.0, 2.4e38),
                                       (0.125, 1e-39), (3e38, 0.0), (3e38, 1.0), (1e-38, 50.0)])
def test_refused(call, scale, cap):
    with pytest.raises(PDAError) as e:
        call(scale, cap)
    assert e.value.status == PDA_EINVAL


def test_a_cap_that_fp32_rounds_to_zero_is_no_missing_cap(call):
    with pytest.raises(ValueError, match="softcap"):
        call(0.1, 1e-50)
