"""run(softcap, alibi_slopes, window) and run_shared_prefix against 64-bit attention."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention
from row_attn_ref import check, make, poison, reference

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def handle(q, k, table, **kw):
    nb, bs, hkv, d = k.shape
    kw.setdefault("max_splits", 4)
    return PagedDecodeAttention(q.shape[1], hkv, d, bs, q.dtype, max_batch=max(1, len(q)),
                                max_blocks_per_seq=table.shape[1], **kw)


def slopes(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float().cuda()


@pytest.mark.parametrize("lens,hq,hkv,d,bs,dtype", [
    ([1], 1, 1, 64, 16, BF),
    ([128], 8, 1, 128, 16, BF),
    ([129, 0, 1, 127, 300], 8, 2, 128, 16, BF),
    ([1000, 17, 0, 2049], 28, 4, 128, 64, HF),
    ([777], 14, 2, 64, 16, BF),
    ([5, 4000], 16, 1, 64, 32, HF),
    ([260, 33], 6, 3, 128, 32, HF),
    ([40000], 4, 1, 128, 16, BF),
])
def test_capped(lens, hq, hkv, d, bs, dtype):
    q, k, v, table, ln = make(lens, hq, hkv, d, bs, dtype, seed=1)
    poison(k, v, table, ln)
    with handle(q, k, table) as a:
        out = a.run(q, k, v, table, ln, 0.2, softcap=5.0)
        assert a.check_device_error() == (0, 0)
    check(out, *reference(q, k, v, table, ln, 0.2, 5.0), f"{lens}")


@pytest.mark.parametrize("softcap,alibi,window", [(0.0, True, 0), (30.0, True, 0), (0.0, False, 100),
                                                  (200.0, False, 0), (1e4, True, 77), (50.0, True, 1),
                                                  (0.0, False, 5000)])
@pytest.mark.parametrize("d,dtype,g", [(128, BF, 4), (64, HF, 7)])
def test_kinds_of_scores(softcap, alibi, window, d, dtype, g):
    lens = [1, 100, 101, 640, 3000, 0]
    q, k, v, table, ln = make(lens, 2 * g, 2, d, 16, dtype, seed=2)
    poison(k, v, table, ln, window)
    sl = slopes(2 * g) if alibi else None
    with handle(q, k, table) as a:
        out = a.run(q, k, v, table, ln, softcap=softcap, alibi_slopes=sl, window=window)
        assert a.check_device_error() == (0, 0)
    check(out, *reference(q, k, v, table, ln, d ** -0.5, softcap, sl, window))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_scales(scale):
    q, k, v, table, ln = make([300, 5], 8, 2, 128, 16, BF, seed=3)
    with handle(q, k, table) as a:
        out = a.run(q, k, v, table, ln, scale, window=250)
        check(out, *reference(q, k, v, table, ln, scale, window=250))
        out = a.run(q, k, v, table, ln, scale, softcap=2.0)
        check(out, *reference(q, k, v, table, ln, scale, 2.0))


@pytest.mark.parametrize("own,prefix,hq,hkv,d,bs,dtype", [
    ([3, 1], 64, 8, 1, 128, 16, BF),                       # one row tile in part
    ([5] * 20 + [300, 1, 129], 640, 16, 2, 128, 16, BF),   # wide
    ([40] * 64, 1024, 16, 2, 64, 32, HF),                  # two whole tiles of 256 rows
    ([7] * 33, 1000, 14, 2, 128, 16, HF),                  # groups of 7, a prefix inside a block
    ([9, 200] * 9, 777, 32, 2, 64, 16, BF),                # groups of 16
    ([2] * 129 + [1], 300, 2, 1, 128, 64, BF),             # groups of 2: 260 rows
    ([1, 2, 3], 5000, 3, 3, 128, 16, BF),                  # groups of 1
])
def test_shared_prefix(own, prefix, hq, hkv, d, bs, dtype):
    lens = [prefix + n for n in own]
    q, k, v, table, ln = make(lens, hq, hkv, d, bs, dtype, groups=[(0, len(own), prefix)], seed=4)
    poison(k, v, table, ln)
    cu = torch.tensor([0, len(own)], dtype=torch.int32, device="cuda")
    pl = torch.tensor([prefix], dtype=torch.int32, device="cuda")
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, cu, pl, 0.15)
        assert a.check_device_error() == (0, 0)
        check(out, *reference(q, k, v, table, ln, 0.15))
        sl = slopes(hq)
        out = a.run_shared_prefix(q, k, v, table, ln, cu, pl, 0.15, softcap=8.0, alibi_slopes=sl)
        check(out, *reference(q, k, v, table, ln, 0.15, 8.0, sl))
