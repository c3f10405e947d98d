"""Decode attention over a block-scaled FP8 cache at the edges of its formats:
one block, queries that need all of fp16's bits, the largest scales."""
import numpy as np
import pytest
import torch

import fp8_cache_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_fp8_block_attn import Problem, check, expect  # noqa: E402


def two_term_residual(x):
    """What two E4M3 terms of x, scaled so that the largest is in [128, 256), leave of it."""
    y = np.asarray(x, np.float64) * 128
    for _ in range(2):
        y = y - ref.decode(ref.encode(y))
    return y / 128


@pytest.mark.parametrize("G,Hkv,D,bs", [(4, 2, 128, 16), (8, 1, 128, 64), (2, 8, 64, 32)])
@pytest.mark.parametrize("blocks", [1, 2])
def test_fp16_queries_keep_their_bits_however_many_blocks(G, Hkv, D, bs, blocks):
    """Half the dimensions of q leave a positive rest after two E4M3 terms, half a negative one,
    and the first of two tokens meets them with large keys of opposite signs: two terms would
    move its logit by about 0.2. Three hold an fp16 value exactly (4 + 4 + 4 bits), so the tolerance is the
    one of exact queries."""
    grid = 1 + np.arange(1024) / 1024  # fp16 values in [1, 2)
    rest = two_term_residual(grid)
    near = grid < 1.25
    hi, lo = grid[near][np.argmax(rest[near])], grid[near][np.argmin(rest[near])]
    p = Problem(31, G, Hkv, D, bs, [2], "fp16", extra_blocks=blocks - 1)
    q = np.where(np.arange(D) < D // 2, hi, lo)
    p.q = torch.from_numpy(np.tile(q, (1, G * Hkv, 1))).to(torch.float16)
    blk = p.table[0, 0]
    p.kc[blk] = 0
    p.kc[blk, 0] = ref.encode(np.where(np.arange(D) < D // 2, 448.0, -448.0))
    p.ks[blk] = 50 / (448 * D / 2 * p.scale)  # 50 from either half
    v = np.ones((bs, Hkv, D)) * 2.0
    v[0] = -2.0
    p.vc[blk], p.vs[blk] = ref.encode(v), 1.0
    p.upload()
    want = expect(p.q.double().numpy(), p.kc, p.vc, p.ks, p.vs, p.table, p.lens, float(np.float32(p.scale)), False)
    moved = p.scale * float(p.ks[blk, 0]) * 448 * (np.abs(two_term_residual(q)).sum())
    assert moved > 0.1
    with p.attn() as attn:
        check(p.run(attn, out_dtype=torch.float32), want, "fp32 out")
        check(p.run(attn), want)


@pytest.mark.parametrize("G,Hkv,D,bs", [(4, 2, 128, 16), (8, 1, 128, 32), (3, 2, 64, 64), (16, 1, 64, 16)])
def test_large_values(G, Hkv, D, bs):
    """V up to nearly 2^121, over one split and several; one token's come out as they are."""
    p = Problem(32, G, Hkv, D, bs, [700, 1, 130, 3], "bf16", spread=0)
    p.vs *= np.float32(2.0 ** 113)
    p.upload()
    want = p.want()
    assert np.abs(want[0]).max() > 2.0 ** 120
    with p.attn() as attn:
        for s in (1, 0, 4):
            check(p.run(attn, num_splits=s, out_dtype=torch.float32), want, f"splits {s}")
        check(p.run(attn), want)


@pytest.mark.parametrize("G,Hkv,D,bs", [(4, 2, 128, 16), (8, 1, 128, 32), (3, 2, 64, 64), (16, 1, 64, 16)])
@pytest.mark.parametrize("e", [120, 100, -52])
def test_large_and_small_keys_against_queries_of_the_other_kind(G, Hkv, D, bs, e):
    """K scales 2^e times the usual ones and queries as much smaller or larger: the usual logits.
    One block's keys are zeros under the largest scale."""
    p = Problem(33, G, Hkv, D, bs, [700, 5, 130], "bf16")
    p.ks *= np.float32(2.0 ** e)
    p.q = (p.q.float() * 2.0 ** -e).to(torch.bfloat16)
    zero = p.table[0, 1]
    p.kc[zero], p.ks[zero] = 0, 2.0 ** 127
    p.upload()
    want = p.want()
    with p.attn() as attn:
        for s in (1, 0):
            check(p.run(attn, num_splits=s, out_dtype=torch.float32), want, f"splits {s}")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_one_block_calls_in_the_per_head_shapes(dt):
    """What the per-head call takes runs with [1, Hkv] scales of a one-block cache as well: a flat
    q and out, a table and lengths with more rows than the batch."""
    p = Problem(34, 4, 8, 128, 16, [13, 7], dt, extra_blocks=0)
    p.kc, p.vc, p.ks, p.vs = p.kc[:1], p.vc[:1], p.ks[:1], p.vs[:1]
    for c in (p.kc, p.vc):
        c[(c & 0x7F) == 0x7F] = 0x30
    p.table[:] = 0
    p.upload()
    want = p.want()
    q, kc, vc, table, lens, scale = p.dev
    out = torch.empty(2, 32 * 128, dtype=q.dtype, device=q.device)
    more = torch.cat([table, table]), torch.cat([lens, lens])
    with p.attn() as attn:
        check(attn.run(q, kc, vc, table, lens, scale, **p.scales), want)
        check(attn.run(q.view(2, -1), kc, vc, table, lens, scale, **p.scales), want, "flat q")
        check(attn.run(q, kc, vc, table, lens, scale, out=out, **p.scales).view(q.shape), want, "flat out")
        check(attn.run(q, kc, vc, *more, scale, **p.scales), want, "more rows")
        assert attn.check_device_error() == (0, 0)
