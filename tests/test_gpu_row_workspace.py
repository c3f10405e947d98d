"""A handle whose memory suffices for run, but not for the partials of scored attention and shared
prefixes, is created, serves run, and refuses those two calls."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PDA_ENOMEM, PDAError, PagedDecodeAttention

pytestmark = pytest.mark.gpu


def test_handle_without_memory_for_the_row_tiled_calls():
    torch.cuda.empty_cache()
    total, d, most = torch.cuda.mem_get_info()[1], 128, 16384
    heads = int(0.28 * total) // (most * (d + 1) * 4)  # run's partials: 28% of the memory; theirs: four times that
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, heads, d, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(2, 16, heads, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    table = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([16, 5], dtype=torch.int32, device="cuda")
    with PagedDecodeAttention(heads, heads, d, 16, torch.bfloat16, max_batch=most, max_blocks_per_seq=1, max_splits=1) as a:
        out = a.run(q, k, v, table, ln, out_dtype=torch.float32)
        for call in (lambda: a.run(q, k, v, table, ln, softcap=5.0),
                     lambda: a.run_shared_prefix(q, k, v, table, ln, ln[:1] * 0, ln[:0])):
            with pytest.raises(PDAError) as e:
                call()
            assert e.value.status == PDA_ENOMEM
        assert a.check_device_error() == (0, 0)
    s = torch.einsum("bhd,bthd->bht", q.float(), k[[1, 0]].float()) * d ** -0.5
    s = s.masked_fill(torch.arange(16, device="cuda") >= ln.long()[:, None, None], float("-inf"))
    want = torch.einsum("bht,bthd->bhd", torch.softmax(s, -1), v[[1, 0]].float())
    # weights within 2^-16 of themselves, 128 products and 16 weights in fp32, |v| < 8: far below 2^-10
    assert float((out - want).abs().max()) < 2.0 ** -10


@pytest.mark.parametrize("splits", [1, 64])
def test_partials_beside_and_within_the_splits(splits):
    """The two calls at the handle's largest batch, between calls of run."""
    from row_attn_ref import check, make, reference
    q, k, v, table, ln = make([700 + i for i in range(48)], 16, 2, 128, 16, torch.bfloat16, [(0, 48, 640)], seed=2)
    cu, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 48], [640]))
    want, capped = reference(q, k, v, table, ln, 0.1), reference(q, k, v, table, ln, 0.1, 4.0)
    with PagedDecodeAttention(16, 2, 128, 16, torch.bfloat16, max_batch=48, max_blocks_per_seq=table.shape[1],
                              max_splits=splits) as a:
        first = a.run(q, k, v, table, ln, 0.1)
        for _ in range(3):
            check(a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.1), *want)
            check(a.run(q, k, v, table, ln, 0.1, softcap=4.0), *capped)
            assert torch.equal(a.run(q, k, v, table, ln, 0.1), first)
