"""Where run(softcap, alibi_slopes, window) and run_shared_prefix can go wrong: empty and padded
sequences, odd groupings, bad ids, growing maxima, large values, capture, streams, refusals."""
import random

import pytest
import torch

from paged_gqa_decode_attention_gb300 import (PDA_EALIAS, PDA_EINVAL, PDA_EUNSUPPORTED, PDAError,
                                              PagedDecodeAttention, rope_axes_kv_write,
                                              rope_pair_axes)
from row_attn_ref import check, make, poison, reference

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def handle(q, k, table, **kw):
    nb, bs, hkv, d = k.shape
    kw.setdefault("max_splits", 1)
    return PagedDecodeAttention(q.shape[1], hkv, d, bs, q.dtype, max_batch=max(1, len(q)),
                                max_blocks_per_seq=table.shape[1], **kw)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def shared(groups, batch):
    """cu_seqs and prefix_lens of groups (first, last, prefix), ascending."""
    cu, pre = [groups[0][0]], []
    for a, z, n in groups:
        if a > cu[-1]:
            cu.append(a)
            pre.append(0)
        cu.append(z)
        pre.append(n)
    return ints(*cu), ints(*pre)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(16, 2, 128, BF), (9, 3, 64, HF), (32, 2, 128, HF)])
def test_groups_with_empty_and_lone_sequences(hq, hkv, d, dtype):
    # two outside, a group whose first sequence is empty (its table row holds no ids), a group of one, a
    # group without a prefix, a wide one with empty rows, one outside behind
    groups = [(2, 6, 200), (6, 7, 100), (7, 10, 0), (10, 45, 600)]
    lens = [50, 0] + [0, 203, 200, 400] + [150] + [1, 2, 300] + [601 + 13 * i for i in range(35)] + [77]
    lens[20] = lens[44] = 0
    q, k, v, table, ln = make(lens, hq, hkv, d, 16, dtype, groups, seed=11)
    table[2], table[20] = -7, 2 ** 30
    poison(k, v, table, ln)
    cu, pre = shared(groups, len(lens))
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.1)
        assert a.check_device_error() == (0, 0)
    check(out, *reference(q, k, v, table, ln, 0.1))
    assert (out[[1, 2, 20, 44]] == 0).all()


@pytest.mark.parametrize("prefix", [10 ** 6, 513, -5, 15])
def test_prefix_lengths_beyond_what_is_shared(prefix):
    lens, groups = [513, 900, 640], [(0, 3, 512)]
    q, k, v, table, ln = make(lens, 8, 2, 128, 16, BF, groups, seed=12)
    poison(k, v, table, ln)
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, ints(0, 3), ints(prefix), 0.1)
    check(out, *reference(q, k, v, table, ln, 0.1))


@pytest.mark.parametrize("cu", [(0, 3, 1), (-1, 2, 4), (0, 2, 9)])
def test_cu_seqs_out_of_order_share_nothing(cu):
    q, k, v, table, ln = make([200, 300, 40, 129], 8, 2, 64, 16, BF, seed=13)
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, ints(*cu), ints(100, 100), 0.2)
        assert a.check_device_error()[0] == 6
        assert a.check_device_error() == (0, 0)
    check(out, *reference(q, k, v, table, ln, 0.2))


def test_no_prefixes_and_no_sequences():
    q, k, v, table, ln = make([200, 30], 8, 2, 64, 16, BF, seed=14)
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, ints(0), ints(), 0.2)
        check(out, *reference(q, k, v, table, ln, 0.2))
        assert a.run(q[:0], k, v, table[:0], ln[:0], softcap=3.0).shape == (0, 8, 64)
        out = a.run(q, k, v, table, torch.zeros_like(ln), window=5)
        assert (out == 0).all()


def test_ids_out_of_range_read_zeros():
    q, k, v, table, ln = make([400, 400, 400], 8, 2, 128, 16, BF, seed=15)
    table[0, 3], table[1, 0], table[2, 24] = len(k), -1, 2 ** 31 - 1
    want = reference(q, k, v, table, ln, 0.1, 6.0)
    with handle(q, k, table) as a:
        check(a.run(q, k, v, table, ln, 0.1, softcap=6.0), *want)
        assert a.check_device_error() == (0, 0)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 128, BF), (24, 2, 64, HF)])
@pytest.mark.parametrize("seqs", [3, 40])  # queries of a tile, and of a wide one
@pytest.mark.parametrize("softcap", [0.0, 6.0])
def test_nan_in_a_query_or_a_key_reaches_its_rows_only(hq, hkv, d, dtype, seqs, softcap):
    lens = [193 + 5 * i for i in range(seqs)]
    q, k, v, table, ln = make(lens, hq, hkv, d, 16, dtype, [(0, seqs, 192)], seed=31)
    want, tol = reference(q, k, v, table, ln, 0.1, softcap)
    nan = torch.zeros(seqs, hq, dtype=torch.bool)
    q[1, 3, 7] = float("nan")
    nan[1, 3] = True
    k[table[0, 12], 0, 1, 5] = float("nan")  # the first sequence's only token of its own
    nan[0, hq // 2:] = True
    cu, pre = ints(0, seqs), ints(192)
    with handle(q, k, table) as a:
        for out in (a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.1, softcap),
                    a.run(q, k, v, table, ln, 0.1, softcap=softcap, window=10 ** 6)):
            assert torch.isnan(out.cpu()[nan]).all()
            check(out.cpu()[~nan], want[~nan], tol[~nan])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("order", [1, -1])
def test_growing_and_falling_scores(dtype, order):
    """The largest score moves at nearly every chunk, or stays far behind: 30 powers of e over the
    context. Wide, narrow and own segments."""
    groups = [(0, 20, 1000), (20, 23, 1000)]
    lens = [1000 + 97 * (i % 7) for i in range(23)] + [1500]
    q, k, v, table, ln = make(lens, 16, 2, 64, 16, dtype, groups, seed=16)
    q.copy_(q.abs())
    pos = torch.zeros(k.shape[:2], device="cuda")
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        pos[table[b].long()[at // 16], at % 16] = at / 1500.0 if order > 0 else 1 - at / 1500.0
    k.copy_((pos[:, :, None, None] * 5.0 + 0.1 * k.float()).to(dtype))
    cu, pre = shared(groups, len(lens))
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.12)
        check(out, *reference(q, k, v, table, ln, 0.12))
        out = a.run(q, k, v, table, ln, 0.12, window=1499)
        check(out, *reference(q, k, v, table, ln, 0.12, window=1499))


def test_values_near_the_largest_stay_finite():
    groups = [(0, 40, 2000)]
    lens = [2000 + 30 * i for i in range(40)] + [3000]
    q, k, v, table, ln = make(lens, 8, 1, 64, 16, BF, groups, seed=17, spread=0.01)
    v.copy_(torch.where(v > 0.5, 3.0e38, 2.0e38))
    cu, pre = shared(groups, len(lens))
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, cu, pre)
        check(out, *reference(q, k, v, table, ln, 64 ** -0.5))


def test_far_places_of_a_large_cache():
    """Blocks beyond 2^32 bytes and 2^31 values."""
    nb, bs, hkv, d = 140000, 16, 8, 128
    k, v = (torch.empty(nb, bs, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    table = (nb - 1 - torch.randperm(60, device="cuda", generator=g)).to(torch.int32).view(3, 20)
    table[1, :10], table[2, :10] = table[0, :10], table[0, :10]
    for t in (k, v):
        t[table.long().flatten()] = torch.randn(60, bs, hkv, d, device="cuda", generator=g).to(BF)
    q = torch.randn(3, 32, d, device="cuda", generator=g).to(BF)
    ln = ints(320, 200, 161)
    rows = table.flatten().long().unique()
    small = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
    small[rows] = torch.arange(len(rows), dtype=torch.int32, device="cuda")
    want = reference(q, k[rows], v[rows], small[table.long()], ln, 0.1)
    with handle(q, k, table) as a:
        check(a.run_shared_prefix(q, k, v, table, ln, ints(0, 3), ints(160), 0.1), *want)


def test_more_sequences_than_threads():
    rng = random.Random(5)
    groups, at = [], 3
    for _ in range(100):
        n = rng.randint(1, 9)
        groups.append((at, at + n, 16 * rng.randint(0, 4)))
        at += n
    lens = [rng.randint(0, 90) for _ in range(at + 2)]
    for a, z, n in groups:
        for b in range(a, z):
            lens[b] = n + rng.randint(1, 40)
    q, k, v, table, ln = make(lens, 4, 2, 64, 16, HF, groups, seed=18)
    cu, pre = shared(groups, len(lens))
    with handle(q, k, table) as a:
        out = a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.2)
        assert a.check_device_error() == (0, 0)
    check(out, *reference(q, k, v, table, ln, 0.2))


@pytest.mark.parametrize("seed", range(12))
def test_drawn(seed):
    rng = random.Random(seed)
    hkv, g, bs = rng.choice([1, 2, 3]), rng.randint(1, 16), rng.choice([16, 32])
    d, dtype = rng.choice([64, 128]), rng.choice([BF, HF])
    groups, at = [], 0
    while at < 30 and rng.random() < 0.8:
        n = rng.choice([1, 2, 5, 17, 40])
        groups.append((at, at + n, rng.choice([0, 5, 100, 777, 1024])))
        at += n
    lens = []
    for a, z, n in groups:
        lens += [n + rng.choice([0, 1, 64, rng.randint(0, 400)]) for _ in range(a, z)]
    lens += [rng.randint(0, 700) for _ in range(rng.randint(0, 4))] or [33]
    q, k, v, table, ln = make(lens, hkv * g, hkv, d, bs, dtype, groups, seed=seed)
    poison(k, v, table, ln)
    cap = rng.choice([0.0, 0.0, 2.0, 300.0])
    sl = torch.linspace(0.3, -0.01, hkv * g).cuda() if rng.random() < 0.4 else None
    with handle(q, k, table) as a:
        if groups:
            cu, pre = shared(groups, len(lens))
            out = a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.2, cap, sl)
            again = a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.2, cap, sl)
            assert torch.equal(out, again)
            assert a.check_device_error() == (0, 0)
            check(out, *reference(q, k, v, table, ln, 0.2, cap, sl))
        w = rng.choice([1, 30, 129, 10 ** 6])
        out = a.run(q, k, v, table, ln, 0.2, softcap=cap, alibi_slopes=sl, window=w)
        check(out, *reference(q, k, v, table, ln, 0.2, cap, sl, w))


def test_captured_with_other_lengths():
    groups = [(0, 12, 320)]
    lens = [320 + 11 * i for i in range(12)]
    q, k, v, table, ln = make(lens, 16, 2, 64, 16, BF, groups, seed=21)
    cu, pre = shared(groups, 12)
    out = torch.empty_like(q)
    with handle(q, k, table) as a:
        a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.2, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.run_shared_prefix(q, k, v, table, ln, cu, pre, 0.2, out=out)
            capped = a.run(q, k, v, table, ln, 0.2, softcap=4.0)
        for cut in (0, 100):
            ln.sub_(cut).clamp_(min=0)
            pre.sub_(cut)
            q.copy_(q.flip(0))
            graph.replay()
            torch.cuda.synchronize()
            check(out, *reference(q, k, v, table, ln, 0.2))
            check(capped, *reference(q, k, v, table, ln, 0.2, 4.0))
        assert a.check_device_error() == (0, 0)


def test_two_handles_on_two_streams():
    sets = []
    for seed in (1, 2):
        lens = [700 + seed * 37 + i for i in range(20)]
        t = make(lens, 16, 2, 128, 16, BF, [(0, 20, 640)], seed=seed)
        sets.append((t, handle(t[0], t[1], t[3]), torch.cuda.Stream()))
    cu, pre = ints(0, 20), ints(640)
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (t, a, s) in enumerate(sets):
            with torch.cuda.stream(s):
                outs[i].append(a.run_shared_prefix(*t, cu, pre, 0.1))
    torch.cuda.synchronize()
    for (t, a, _), got in zip(sets, outs):
        check(got[0], *reference(*t, 0.1))
        assert all(torch.equal(got[0], o) for o in got)
        assert a.check_device_error() == (0, 0)
        a.close()


def test_refusals():
    q, k, v, table, ln = make([200, 300], 8, 2, 128, 16, BF, seed=22)
    cu, pre = ints(0, 2), ints(100)
    fine = dict(q=q, k_cache=k, v_cache=v, block_table=table, context_lens=ln)
    with handle(q, k, table) as a:
        def status(want, f, **kw):
            with pytest.raises(PDAError) as e:
                f(**{**fine, **kw})
            assert e.value.status == want, e.value

        for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                   dict(window=-1), dict(softcap=1e-40), dict(softcap=1.0, scale=float("inf"))):
            status(PDA_EINVAL, a.run, **kw)
        status(PDA_EALIAS, a.run, window=3, out=q)
        many = torch.zeros(130, dtype=torch.int32, device="cuda")
        status(PDA_EUNSUPPORTED, a.run_shared_prefix, cu_seqs=many, prefix_lens=many[1:])
        for kw in (dict(num_splits=2), dict(out_dtype=torch.float32), dict(k_scale=ln.float()),
                   dict(alibi_slopes=torch.zeros(7, device="cuda")),
                   dict(alibi_slopes=torch.zeros(8, device="cuda", dtype=BF)),
                   dict(alibi_slopes=torch.zeros(8)), dict(q=q[:, :4]), dict(q=q.half()),
                   dict(block_table=table[:1]), dict(context_lens=ln.long()),
                   dict(q=torch.cat([q, q], 2)[:, :, :128]), dict(out=torch.empty_like(q[:1]))):
            with pytest.raises(ValueError):
                a.run(**{**fine, **kw}, window=9)
        for kw in (dict(cu_seqs=None, prefix_lens=pre), dict(cu_seqs=cu, prefix_lens=None),
                   dict(cu_seqs=cu, prefix_lens=ints(1, 2)), dict(cu_seqs=cu.long(), prefix_lens=pre),
                   dict(cu_seqs=cu.cpu(), prefix_lens=pre)):
            with pytest.raises(ValueError):
                a.run_shared_prefix(**fine, **kw)
        out = a.run(**fine, window=9)  # and goes on
        check(out, *reference(q, k, v, table, ln, 128 ** -0.5, window=9))


@pytest.mark.parametrize("kw", [dict(head_dim=256, num_q_heads=4), dict(kv_fp8=True, num_q_heads=8)])
def test_geometries_without_row_calls(kw):
    d = kw.get("head_dim", 128)
    dt = torch.float8_e4m3fn if kw.get("kv_fp8") else BF
    k = torch.zeros(8, 16, 2, d, device="cuda").to(dt)
    q = torch.zeros(1, kw["num_q_heads"], d, dtype=BF, device="cuda")
    a = PagedDecodeAttention(num_kv_heads=2, block_size=16, max_batch=1, max_blocks_per_seq=4,
                             **{"head_dim": 128, **kw})
    with a, pytest.raises(PDAError) as e:
        a.run(q, k, k.clone(), ints(0, 1, 2, 3).view(1, 4), ints(30), softcap=5.0)
    assert e.value.status == PDA_EUNSUPPORTED


def test_prompt_written_with_axes_then_sampled_from():
    """A prompt with image tokens is written to the cache with positions on three axes, four
    samples share it, and each step writes one more token and attends to everything."""
    hq, hkv, d, bs, prompt, samples = 8, 2, 64, 16, 300, 4
    g = torch.Generator().manual_seed(3)
    axis = rope_pair_axes((12, 10, 10), interleaved=True)
    inv = 1e4 ** (-torch.arange(d // 2).double() / (d // 2))
    ang = torch.arange(400).double()[:, None] * inv
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    k, v = (torch.zeros(60, bs, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    ids = torch.randperm(60, generator=g).to(torch.int32).cuda()
    table = torch.zeros(samples, 22, dtype=torch.int32, device="cuda")
    whole = prompt // bs
    table[:, :whole] = ids[:whole]
    for s in range(samples):
        table[s, whole:] = ids[whole + s * 4:whole + s * 4 + 22 - whole]

    def write(rows, pos, slots):
        qkv = torch.randn(rows, hq + 2 * hkv, d, generator=g).to(BF).cuda()
        return rope_axes_kv_write(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots, cs, k, v, axis)

    at = torch.arange(prompt, device="cuda")
    pos = torch.stack([at // 20, at // 5 % 4, at % 5]).to(torch.int32)
    write(prompt, pos, table[0].long()[at // bs] * bs + at % bs)
    tail = table[:, whole].long()  # the prompt's last tokens, copied to every sample's own block
    k[tail[1:]], v[tail[1:]] = k[tail[0]].clone(), v[tail[0]].clone()
    cu, pre = ints(0, samples), ints(prompt)
    with PagedDecodeAttention(hq, hkv, d, bs, max_batch=samples, max_blocks_per_seq=22, max_splits=2) as a:
        for step in range(6):
            n = prompt + step
            slots = table[:, n // bs].long() * bs + n % bs
            q = write(samples, torch.full((3, samples), 20 + step, dtype=torch.int32, device="cuda"), slots)
            ln = torch.full((samples,), n + 1, dtype=torch.int32, device="cuda")
            out = a.run_shared_prefix(q, k, v, table, ln, cu, pre, softcap=20.0)
            check(out, *reference(q, k, v, table, ln, d ** -0.5, 20.0), f"step {step}")
