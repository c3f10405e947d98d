"""append_kv_fp8 and rope_append_kv_fp8 with cu_rows that do not ascend or leave the
input: code 1, the sequence is not appended, every block of the others is
written in full or left alone, and nothing else is written."""
import numpy as np
import pytest
import torch

import fp8_cache_ref as ref
from paged_gqa_decode_attention_gb300 import append_kv_fp8, rope_append_kv_fp8

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_fp8_cache import Cache, dev, rows_of, tables  # noqa: E402

CASES = [  # cu_rows, lengths, rows, block size
    ([0, 10, 8, 25], [20, 30, 40], 25, 16),
    ([0, 40, 8, 60], [50, 40, 60], 60, 16),
    ([320, 480, 0, 16], [160, 16, 16], 480, 16),
    ([100, 0, 100], [100, 130], 100, 32),
    ([-20, 10, 30], [60, 70], 30, 16),
    ([0, 30, 200], [31, 170], 60, 64),
    ([0, 70, 10, 80, 20, 90, 85], [70, 70, 80, 70, 75, 71], 90, 32),
]


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("cu,lens,T,bs", CASES)
def test_descending_rows(cu, lens, T, bs, rope):
    gen = torch.Generator().manual_seed(T)
    rng = np.random.default_rng(T)
    Hkv, D, B = 2, 64, len(lens)
    bad = {b for b in range(B) if cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > T}
    assert bad
    cache = Cache(T, sum(-(-x // bs) for x in lens) + 2, bs, Hkv, D)
    before = [x.copy() for x in (cache.k, cache.v, cache.ks, cache.vs)]
    table = tables(rng, lens, bs, cache.k.shape[0])
    x = rows_of(gen, T, 2 * Hkv, D, "bf16")
    for b in set(range(B)) - bad:
        for rows, c, s in ((x[:, :Hkv], cache.k, cache.ks), (x[:, Hkv:], cache.v, cache.vs)):
            ref.append(rows.double().numpy(), c, s, table[b:b + 1], lens[b:b + 1], cu[b:b + 2])
    xd = x.to(cache.dev[0].device)
    err = torch.zeros(2, dtype=torch.int32, device=xd.device)
    args = (*cache.dev, dev(table), dev(np.array(lens), torch.int32), dev(np.array(cu), torch.int64))
    if rope:  # rotations by no angle: the same bytes
        q = rows_of(gen, T, 4, D, "bf16").to(xd.device)
        q_in = q.clone()
        cos_sin = torch.cat([torch.ones(8, D // 2), torch.zeros(8, D // 2)], 1).to(xd.device)
        rope_append_kv_fp8(q, xd[:, :Hkv], xd[:, Hkv:], torch.zeros(T, dtype=torch.int32, device=xd.device), cos_sin,
                           *args, q_out=q, err=err)
        assert torch.equal(q, q_in)
    else:
        append_kv_fp8(xd[:, :Hkv], xd[:, Hkv:], *args, err=err)
    torch.cuda.synchronize()
    code, which = err.tolist()
    assert code == 1 and which in bad
    kc, vc, ks, vs = [t.view(torch.uint8).cpu().numpy() if t.dim() == 4 else t.cpu().numpy() for t in cache.dev]
    for got, got_s, old, old_s, new, new_s in ((kc, ks, before[0], before[2], cache.k, cache.ks),
                                               (vc, vs, before[1], before[3], cache.v, cache.vs)):
        for blk in range(got.shape[0]):
            for h in range(Hkv):
                left = np.array_equal(got[blk, :, h], old[blk, :, h]) and got_s[blk, h] == old_s[blk, h]
                full = np.array_equal(got[blk, :, h], new[blk, :, h]) and got_s[blk, h] == new_s[blk, h]
                assert left or full, (blk, h)
