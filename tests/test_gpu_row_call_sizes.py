"""Both sides of the limit on batch * num_kv_heads * table width of scored attention and of shared
prefixes: short contexts behind a wide table are served up to it, and a window is what counts."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PDA_EUNSUPPORTED, PDAError, PagedDecodeAttention
from row_attn_ref import check, reference

pytestmark = pytest.mark.gpu
B, HKV, BS, D = 1024, 32, 64, 64  # chunks n of 128 tokens: served up to 8 n + 6 <= 2^30 / 2^15, n = 4095


@pytest.mark.parametrize("blocks,window,prefixes,served", [
    (8190, 0, False, True), (8192, 0, False, False),
    (20000, 1, False, True), (20000, 4095 * 128 - 63, False, True), (20000, 4095 * 128 - 62, False, False),
    (8186, 0, True, True), (8188, 0, True, False),
])
def test_wide_tables(blocks, window, prefixes, served):
    g = torch.Generator(device="cuda").manual_seed(blocks)
    q = torch.randn(B, HKV, D, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(16, BS, HKV, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    table = torch.zeros(B, blocks, dtype=torch.int32, device="cuda")
    table[:, 1] = torch.arange(B, device="cuda") % 16
    ln = (torch.arange(B, device="cuda") % 121).int()
    cu, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, B], [64]))
    with PagedDecodeAttention(HKV, HKV, D, BS, max_batch=B, max_blocks_per_seq=blocks, max_splits=1) as a:
        def run():
            if prefixes:
                return a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.2)
            return a.run(q, k, v, table, ln, 0.2, softcap=4.0, window=window)
        if not served:
            with pytest.raises(PDAError) as e:
                run()
            assert e.value.status == PDA_EUNSUPPORTED
            return
        out = run()
        assert a.check_device_error() == (0, 0)
    some = torch.tensor([0, 1, 63, 64, 120, 500, B - 1], device="cuda")
    check(out[some], *reference(q[some], k, v, table[some], ln[some], 0.2, 0.0 if prefixes else 4.0, None, window))
