"""rope_axes_kv_write against the formula in float64, rounded once: bit for bit, the whole caches."""
import pytest
import torch

from paged_gqa_decode_attention_gb300 import rope_axes_kv_write, rope_kv_write, rope_pair_axes

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def round16(x, dtype):
    """float64 rounded once to a 16-bit type (a cast would round to 32 bits first)."""
    digits, low = (8, -125) if dtype == BF else (11, -13)
    _, e = torch.frexp(x)
    step = torch.exp2((e.clamp(min=low) - digits).double())
    return (torch.round(x / step) * step).to(dtype)


def turned(x, positions, cs, axis, neox):
    rot = cs.shape[1]
    half, y = rot // 2, x.double().clone()
    for j, a in enumerate(axis):
        i, k = (j, j + half) if neox else (2 * j, 2 * j + 1)
        row = cs.double()[positions[a].long()]
        c, s = row[:, j, None], row[:, half + j, None]
        p, q = x[..., i].double(), x[..., k].double()
        y[..., i], y[..., k] = p * c - q * s, q * c + p * s
    return round16(y, x.dtype)


def inputs(t, hq, hkv, d, rot, dtype, axes, bs=16, seed=0, top=500):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(t, hq + 2 * hkv, d, generator=g).to(dtype).cuda()
    pos = torch.randint(0, top, (axes, t), generator=g).to(torch.int32).cuda()
    inv = 1e4 ** (-torch.arange(rot // 2).double() / max(1, rot // 2))
    ang = torch.arange(top).double()[:, None] * inv
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    nb = -(-t // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:t].cuda()
    kc, vc = (torch.randn(nb, bs, hkv, d, generator=g).to(dtype).cuda() for _ in range(2))
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots, cs, kc, vc


def compare(args, axis, neox, skip=(), **kw):
    q, k, v, pos, slots, cs, kc, vc = args
    want_q, want_k = turned(q, pos, cs, axis, neox), kc.clone()
    want_v = vc.clone()
    keep = torch.tensor([i for i in range(len(q)) if i not in skip], dtype=torch.long, device="cuda")
    at = keep[slots[keep] >= 0]
    want_k.flatten(0, 1)[slots[at]] = turned(k, pos, cs, axis, neox)[at]
    want_v.flatten(0, 1)[slots[at]] = v[at]
    got = rope_axes_kv_write(q, k, v, pos, slots, cs, kc, vc, axis, neox=neox, **kw)
    torch.cuda.synchronize()
    for name, a, b in (("q", got[keep], want_q[keep]), ("k", kc, want_k), ("v", vc, want_v)):
        assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16)), name


@pytest.mark.parametrize("t,hq,hkv,d,rot,dtype,neox,sections,mixed", [
    (1, 14, 2, 64, 64, BF, True, (16, 8, 8), False),
    (33, 14, 2, 64, 64, HF, True, (12, 10, 10), True),
    (700, 32, 8, 128, 128, BF, True, (16, 24, 24), False),
    (301, 28, 4, 128, 64, HF, False, (10, 11, 11), True),
    (65, 3, 1, 16, 16, BF, False, (3, 5), False),
    (40, 4, 2, 256, 128, BF, True, (1, 20, 30, 13), True),
    (17, 4, 4, 64, 32, HF, True, (16,), False),
])
def test_axes(t, hq, hkv, d, rot, dtype, neox, sections, mixed):
    axis = rope_pair_axes(sections, mixed)
    assert len(axis) == rot // 2
    compare(inputs(t, hq, hkv, d, rot, dtype, len(sections), seed=t), axis, neox)


def test_equal_positions_are_one_axis():
    q, k, v, pos, slots, cs, kc, vc = inputs(100, 8, 2, 128, 128, BF, 3, seed=5)
    pos[1:] = pos[0]
    kc2, vc2 = kc.clone(), vc.clone()
    a = rope_axes_kv_write(q, k, v, pos, slots, cs, kc, vc, rope_pair_axes((20, 22, 22), True))
    b = rope_kv_write(q, k, v, pos[0].contiguous(), slots, cs, kc2, vc2)
    assert torch.equal(a, b) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_bad_positions_and_slots():
    args = inputs(50, 8, 2, 64, 64, BF, 3, seed=6)
    pos, slots = args[3], args[4]
    pos[2, 7] = 500   # behind the table, on one axis only
    pos[0, 30] = -1
    slots[11] = -1    # no cache write
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    fine = args[3].clamp(0, 499)
    q, k, v, _, _, cs, kc, vc = args
    kc2, vc2 = kc.clone(), vc.clone()
    out = torch.full((50, 8, 64), 3.0, dtype=BF, device="cuda")
    got = rope_axes_kv_write(q, k, v, pos, slots, cs, kc, vc, rope_pair_axes((12, 10, 10)), q_out=out, err=err)
    torch.cuda.synchronize()
    assert err[0] == 4 and int(err[1]) in (7, 30)
    want = turned(q, fine, cs, rope_pair_axes((12, 10, 10)), True)
    for i in range(50):
        if i in (7, 30):
            assert (got[i] == 3).all()
        else:
            assert torch.equal(got[i], want[i])
        if i in (7, 30, 11):
            continue
        kc2.flatten(0, 1)[slots[i]] = turned(k, fine, cs, rope_pair_axes((12, 10, 10)), True)[i]
        vc2.flatten(0, 1)[slots[i]] = v[i]
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_in_place():
    args = inputs(90, 8, 2, 64, 64, HF, 3, seed=8)
    axis = rope_pair_axes((12, 10, 10), True)
    q = args[0]
    want = turned(q, args[3], args[5], axis, True)
    got = rope_axes_kv_write(*args, axis, q_out=q)
    assert got is q and torch.equal(q, want)


def test_captured():
    args = inputs(64, 14, 2, 64, 64, BF, 3, seed=9)
    axis = rope_pair_axes((12, 10, 10))
    out = torch.empty(64, 14, 64, dtype=BF, device="cuda")
    rope_axes_kv_write(*args, axis, q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope_axes_kv_write(*args, axis, q_out=out)
    args[3].copy_(args[3].flip(1))
    args[0].copy_(args[0].flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, turned(args[0], args[3], args[5], axis, True))
