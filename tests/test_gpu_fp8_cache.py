"""GPU parity of the block-scaled FP8 cache: appending (with and without
rotary positions) and reading back, against the 64-bit reference. Scales are
powers of two, so every comparison is exact: the whole caches (the written
bytes and every byte the call must leave alone), the scales, q_out."""
import numpy as np
import pytest
import torch

import fp8_cache_ref as ref
import oracle
from paged_gqa_decode_attention_gb300 import (append_kv_fp8, copy_blocks, gather_kv_fp8,
                                              rope_append_kv_fp8, rope_kv_write, workloads)

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda", torch.cuda.current_device())
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
FP8 = torch.float8_e4m3fn


class Cache:
    """A random block-scaled cache on the GPU and its copy for the reference."""

    def __init__(self, seed, num_blocks, bs, Hkv, D):
        rng = np.random.default_rng(seed)
        self.k = rng.integers(0, 256, (num_blocks, bs, Hkv, D), dtype=np.uint8)
        self.v = rng.integers(0, 256, (num_blocks, bs, Hkv, D), dtype=np.uint8)
        for x in (self.k, self.v):
            x[(x & 0x7F) == 0x7F] = 0  # no NaN codes
        self.ks = np.exp2(rng.integers(-8, 3, (num_blocks, Hkv))).astype(np.float32)
        self.vs = np.exp2(rng.integers(-8, 3, (num_blocks, Hkv))).astype(np.float32)
        self.upload()

    def upload(self):
        self.dev = [torch.from_numpy(self.k.copy()).to(DEV).view(FP8),
                    torch.from_numpy(self.v.copy()).to(DEV).view(FP8),
                    torch.from_numpy(self.ks.copy()).to(DEV), torch.from_numpy(self.vs.copy()).to(DEV)]

    def check(self, what=""):
        torch.cuda.synchronize()
        kc, vc, ks, vs = self.dev
        np.testing.assert_array_equal(ks.cpu().numpy(), self.ks, err_msg=f"{what}: k_scale")
        np.testing.assert_array_equal(vs.cpu().numpy(), self.vs, err_msg=f"{what}: v_scale")
        for name, got, want in (("k", kc, self.k), ("v", vc, self.v)):
            got = got.view(torch.uint8).cpu().numpy()
            nan = (want & 0x7F) == 0x7F
            np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan, err_msg=f"{what}: NaN of {name}")
            np.testing.assert_array_equal(got[~nan], want[~nan], err_msg=f"{what}: {name}_cache")


def tables(rng, lens, bs, num_blocks, width=None):
    width = width or max(1, max(-(-int(x) // bs) for x in lens))
    order = rng.permutation(num_blocks)
    t = np.full((len(lens), width), -7, np.int32)  # entries past a sequence are never read
    at = 0
    for b, x in enumerate(lens):
        n = -(-int(x) // bs)
        t[b, :n] = order[at:at + n]
        at += n
    return t


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t if dtype is None else t.to(dtype)


def rows_of(gen, T, H, D, dt, spread=2.0):
    x = torch.randn(T, H, D, generator=gen) * torch.exp2(spread * torch.randn(T, H, 1, generator=gen))
    return x.to(DT[dt])


BEFORE = [0, 1, 5, 15, 16, 31, 63, 64, 100, 47, 14, 0]
NEW = [1, 1, 0, 2, 1, 2, 70, 64, 33, 17, 3, 130]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 8, 9])
def test_append_geometries(dt, D, bs, Hkv):
    """Ragged appends: from inside blocks and at their borders, none, one, two rows across a
    border, several blocks; rows before the first and behind the last sequence are not read."""
    gen = torch.Generator().manual_seed(bs + D + Hkv)
    rng = np.random.default_rng(bs * D + Hkv)
    lens = np.array(BEFORE) + np.array(NEW)
    cu = np.concatenate([[3], 3 + np.cumsum(NEW)])
    T = int(cu[-1]) + 5
    cache = Cache(Hkv, sum(-(-int(x) // bs) for x in lens) + 3, bs, Hkv, D)
    table = tables(rng, lens, bs, cache.k.shape[0], width=20)
    kv = rows_of(gen, T, 2 * Hkv, D, dt)
    kv[:3], kv[int(cu[-1]):] = float("nan"), float("inf")
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    ref.append(k.double().numpy(), cache.k, cache.ks, table, lens, cu)
    ref.append(v.double().numpy(), cache.v, cache.vs, table, lens, cu)
    fused = kv.to(DEV)
    err = torch.zeros(2, dtype=torch.int32, device=DEV)
    append_kv_fp8(fused[:, :Hkv], fused[:, Hkv:], *cache.dev, dev(table), dev(lens, torch.int32),
                  dev(cu, torch.int64), err=err)
    cache.check(f"{dt} D{D} bs{bs} Hkv{Hkv}")
    assert err.tolist() == [0, 0]


@pytest.mark.parametrize("bs,D", [(16, 64), (32, 128), (64, 128)])
def test_append_token_by_token_with_growing_scales(bs, D):
    """One token a call, sizes that grow by factors: blocks are requantised again and again, down
    into E4M3's subnormals, and start anew at every border."""
    rng = np.random.default_rng(bs)
    B, Hkv, steps = 3, 2, 70
    cache = Cache(7, 16, bs, Hkv, D)
    cache.ks[:], cache.vs[:] = np.nan, -1.0  # never read: every block is started by a call
    cache.upload()
    order = rng.permutation(16)
    table = np.zeros((B, 5), np.int32)
    for b in range(B):
        table[b] = order[b * 5:b * 5 + 5]
    dt = dev(table)
    for t in range(steps):
        x = (rng.standard_normal((B, 2 * Hkv, D)) * 2.0 ** ((t % 23) * 0.7 - 6)).astype(np.float32)
        x = torch.from_numpy(x).to(torch.bfloat16)
        lens = np.array([t + 1, t + 1 + bs // 2, min(t + 1, 3)])
        if t == 0:
            lens[1] = 1 + bs // 2
        n = np.array([1, 1, 1 if t < 3 else 0])
        cu = np.concatenate([[0], np.cumsum(n)])
        T = int(cu[-1])
        k, v = x[:T, :Hkv], x[:T, Hkv:]
        ref.append(k.double().numpy(), cache.k, cache.ks, table, lens, cu)
        ref.append(v.double().numpy(), cache.v, cache.vs, table, lens, cu)
        append_kv_fp8(k.to(DEV).contiguous(), v.to(DEV).contiguous(), *cache.dev, dt,
                      dev(lens, torch.int32), dev(cu, torch.int64))
    cache.check()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_special_values(dt):
    """Zeros, negative zeros, infinities, NaN, subnormals, the largest values, E4M3 midpoints."""
    gen = torch.Generator().manual_seed(3)
    Hkv, D, bs = 4, 64, 16
    info = torch.finfo(DT[dt])
    x = rows_of(gen, 96, 2 * Hkv, D, dt)
    x[0:16] = 0.0
    x[5, :, ::3] = -0.0
    x[17, 0, 5], x[18, 1, 6], x[19, 2, 7] = float("inf"), float("-inf"), float("nan")
    x[20:30, 3] = float("nan")
    x[16:32, 5] = float("inf")          # a tile with nothing finite
    x[32, :, :] = info.max
    x[33, :, :] = -info.max
    x[48:64] = torch.randn(16, 2 * Hkv, D, generator=gen).to(DT[dt]) * info.tiny * 0.25
    mid = torch.tensor((ref.E4M3[:126] + ref.E4M3[1:127]) / 2)[:D].to(DT[dt])
    x[64:80] = mid
    x[64:80, :, 0] = 448.0              # scale 1, so the midpoints are ties
    x[80:96, :, 0] = 449.0
    lens, cu = np.array([96]), np.array([0, 96])
    cache = Cache(1, 8, bs, Hkv, D)
    table = np.array([[5, 2, 7, 0, 1, 3]], np.int32)
    ref.append(x[:, :Hkv].double().numpy(), cache.k, cache.ks, table, lens, cu)
    ref.append(x[:, Hkv:].double().numpy(), cache.v, cache.vs, table, lens, cu)
    xd = x.to(DEV)
    append_kv_fp8(xd[:, :Hkv], xd[:, Hkv:], *cache.dev, dev(table), dev(lens, torch.int32),
                  dev(cu, torch.int64))
    cache.check(dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_append_every_scale_exponent(dt):
    """One block per power of two between the type's extremes: scales from the smallest (2^-60, or
    what the type's subnormals ask for) to the largest, behind old scales that are larger too."""
    gen = torch.Generator().manual_seed(13)
    Hkv, D, bs = 1, 64, 16
    lo, hi = (-133, 127) if dt == "bf16" else (-24, 15)
    exps = list(range(lo, hi + 1))
    B = len(exps)
    unit = torch.rand(B, bs, 2 * Hkv, D, generator=gen, dtype=torch.float64) * 2 - 1
    # every block spans its scale's whole range down to far below E4M3's smallest step
    small = torch.exp2(-torch.randint(0, 24, unit.shape, generator=gen).double())
    x = (unit * small * torch.exp2(torch.tensor(exps).double())[:, None, None, None]).to(DT[dt])
    x = x.reshape(B * bs, 2 * Hkv, D)
    cache = Cache(11, B, bs, Hkv, D)
    table = np.arange(B, dtype=np.int32)[:, None]
    lens, cu = np.full(B, bs), bs * np.arange(B + 1)
    def both(rows, lens, cu):
        ref.append(rows[:, :Hkv].double().numpy(), cache.k, cache.ks, table, lens, cu)
        ref.append(rows[:, Hkv:].double().numpy(), cache.v, cache.vs, table, lens, cu)
        d = rows.to(DEV)
        append_kv_fp8(d[:, :Hkv], d[:, Hkv:], *cache.dev, dev(table), dev(lens, torch.int32),
                      dev(cu, torch.int64))
        cache.check(f"{dt} {lens[0]}")

    both(x, lens, cu)
    # a second token behind a first one whose scale is 2^7 times larger
    first = x.reshape(B, bs, 2 * Hkv, D)[:, 0].double() * 128
    both(first.clamp(-torch.finfo(DT[dt]).max, torch.finfo(DT[dt]).max).to(DT[dt]), np.full(B, 1), np.arange(B + 1))
    both(x.reshape(B, bs, 2 * Hkv, D)[:, 1].contiguous(), np.full(B, 2), np.arange(B + 1))


def test_append_behind_foreign_scales():
    """Blocks written by another quantiser: scales that are no powers of two, zero, negative, NaN,
    infinite, subnormal."""
    gen = torch.Generator().manual_seed(4)
    Hkv, D, bs, B = 2, 128, 32, 8
    cache = Cache(2, B, bs, Hkv, D)
    foreign = np.array([0.013, 3.7, 0.0, -2.0, np.nan, np.inf, 1e-40, 3.0e38], np.float32)
    cache.ks[:], cache.vs[:] = foreign[:, None], foreign[::-1][:, None]
    cache.upload()
    table = np.arange(B, dtype=np.int32)[:, None]
    lens, cu = np.array([9 + b for b in range(B)]), 2 * np.arange(B + 1)
    x = rows_of(gen, 2 * B, 2 * Hkv, D, "bf16", spread=0.5)
    ref.append(x[:, :Hkv].double().numpy(), cache.k, cache.ks, table, lens, cu)
    ref.append(x[:, Hkv:].double().numpy(), cache.v, cache.vs, table, lens, cu)
    xd = x.to(DEV)
    append_kv_fp8(xd[:, :Hkv], xd[:, Hkv:], *cache.dev, dev(table), dev(lens, torch.int32),
                  dev(cu, torch.int64))
    cache.check()


def test_append_many_sequences():
    """More sequences than one search round covers, most with one row, some with none."""
    rng = np.random.default_rng(5)
    gen = torch.Generator().manual_seed(5)
    B, bs, Hkv, D = 1500, 16, 1, 64
    before = rng.integers(0, 40, B)
    new = rng.choice([0, 1, 1, 1, 2, 20], B)
    lens, cu = before + new, np.concatenate([[0], np.cumsum(new)])
    cache = Cache(3, int(sum(-(-lens // bs))) + 1, bs, Hkv, D)
    table = tables(rng, lens, bs, cache.k.shape[0])
    x = rows_of(gen, int(cu[-1]), 2, D, "bf16")
    ref.append(x[:, :1].double().numpy(), cache.k, cache.ks, table, lens, cu)
    ref.append(x[:, 1:].double().numpy(), cache.v, cache.vs, table, lens, cu)
    xd = x.to(DEV)
    append_kv_fp8(xd[:, :1], xd[:, 1:], *cache.dev, dev(table), dev(lens, torch.int32),
                  dev(cu, torch.int64))
    cache.check()


@pytest.mark.parametrize("what", ["block", "negative_block", "long", "short", "rows", "descending"])
def test_append_flags_and_skips_bad_sequences(what):
    gen = torch.Generator().manual_seed(6)
    bs, Hkv, D, B = 16, 2, 64, 3
    lens, cu = np.array([20, 30, 40]), np.array([0, 10, 15, 25])
    cache = Cache(4, 8, bs, Hkv, D)
    table = np.array([[0, 1, 2], [3, 4, 4], [5, 6, 7]], np.int32)
    x = rows_of(gen, 25, 2 * Hkv, D, "bf16")
    bad_table, bad_lens, bad_cu, code = table.copy(), lens.copy(), cu.copy(), 1
    T = 25
    ok = [0, 2]
    if what == "block":
        bad_table[1, 1], code = 8, 2
    elif what == "negative_block":
        bad_table[1, 1], code = -1, 2
    elif what == "long":
        bad_lens[1] = 49
    elif what == "short":
        bad_lens[1] = 4
    elif what == "rows":  # the last sequence's rows run past num_rows
        T, ok = 20, [0, 1]
    else:
        bad_cu[2] = 8     # sequence 1 has -2 rows; sequence 2 starts at row 8
    for b in ok:
        for rows, c, s in ((x[:, :Hkv], cache.k, cache.ks), (x[:, Hkv:], cache.v, cache.vs)):
            ref.append(rows.double().numpy(), c, s, table[b:b + 1], bad_lens[b:b + 1],
                       bad_cu[b:b + 2])
    xd = x.to(DEV)[:T]
    err = torch.zeros(2, dtype=torch.int32, device=DEV)
    append_kv_fp8(xd[:, :Hkv], xd[:, Hkv:], *cache.dev, dev(bad_table), dev(bad_lens, torch.int32),
                  dev(bad_cu, torch.int64), err=err)
    if what == "descending":  # what the ascending rest writes is not specified; nothing else is
        torch.cuda.synchronize()
        assert err.tolist()[0] in (0, 1)
    else:
        cache.check(what)
        assert err.tolist() == [code, 2 if what == "rows" else 1]


def test_append_past_4_gib():
    """Blocks whose byte offset exceeds 2^32."""
    gen = torch.Generator().manual_seed(7)
    bs, Hkv, D = 64, 8, 128
    nb = (1 << 32) // (bs * Hkv * D) + 6
    kc = torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    ks = torch.ones(nb, Hkv, device=DEV)
    vs = torch.ones(nb, Hkv, device=DEV)
    x = rows_of(gen, 70, 2 * Hkv, D, "fp16")
    small = Cache(0, 2, bs, Hkv, D)
    small.k[:], small.v[:], small.ks[:], small.vs[:] = 0, 0, 1, 1
    lens, cu = np.array([70]), np.array([0, 70])
    ref.append(x[:, :Hkv].double().numpy(), small.k, small.ks, [[0, 1]], lens, cu)
    ref.append(x[:, Hkv:].double().numpy(), small.v, small.vs, [[0, 1]], lens, cu)
    xd = x.to(DEV)
    table = dev(np.array([[nb - 2, nb - 1]], np.int32))
    append_kv_fp8(xd[:, :Hkv], xd[:, Hkv:], kc, vc, ks, vs, table, dev(lens, torch.int32),
                  dev(cu, torch.int64))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(kc[-2:].cpu().numpy(), small.k)
    np.testing.assert_array_equal(vc[-2:].cpu().numpy(), small.v)
    np.testing.assert_array_equal(ks[-2:].cpu().numpy(), small.ks)
    assert int(kc[:-2].amax()) == 0 and int(vc[:-2].amax()) == 0
    k, v = gather_kv_fp8(kc, vc, ks, vs, table, dev(lens, torch.int32), dtype=torch.float32)
    np.testing.assert_array_equal(k.double().cpu().numpy(),
                                  ref.gather(small.k, small.ks, [[0, 1]], lens)[0])
    np.testing.assert_array_equal(v.double().cpu().numpy(),
                                  ref.gather(small.v, small.vs, [[0, 1]], lens)[0])
    del kc, vc
    torch.cuda.empty_cache()


# ------------------------------ with rotary positions ------------------------------

ORACLE_DT = {"bf16": oracle.BF16, "fp16": oracle.FP16}


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def from_bits(a, dt):
    return torch.from_numpy(a.view(np.int16).copy()).view(DT[dt])


def rope_ref(q, k, v, positions, cos_sin, neox, dt):
    """Rotated q and k as 16-bit tensors, from the FP64 oracle; bad positions give live = False."""
    T, Hkv, D = k.shape
    qo, kc, _ = oracle.rope_kv_write(bits(q), bits(k), bits(v), positions, np.arange(T, dtype=np.int64),
                                     cos_sin, cos_sin.shape[1], neox, ORACLE_DT[dt],
                                     np.zeros((T, 1, Hkv, D), np.uint16), np.zeros((T, 1, Hkv, D), np.uint16),
                                     q_out=None)
    return from_bits(qo.reshape(q.shape), dt), from_bits(kc.reshape(k.shape), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("geom", [(14, 2, 64, 64, 16), (32, 8, 128, 128, 16), (7, 7, 128, 64, 32),
                                  (3, 1, 64, 16, 64), (5, 5, 64, 32, 32), (16, 1, 128, 128, 64),
                                  (4, 2, 128, 0, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_append(dt, neox, geom, in_place):
    Hq, Hkv, D, rot, bs = geom
    gen = torch.Generator().manual_seed(Hq + D)
    rng = np.random.default_rng(Hq * rot + bs)
    lens = np.array(BEFORE) + np.array(NEW)
    cu = np.concatenate([[2], 2 + np.cumsum(NEW)])
    T = int(cu[-1]) + 4
    qkv = rows_of(gen, T, Hq + 2 * Hkv, D, dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    max_pos = 5000
    positions = rng.integers(0, max_pos, T).astype(np.int32)
    cos_sin = workloads.rope_cos_sin(max_pos, rot, 10000.0).numpy() if rot else np.zeros((max_pos, 0), np.float32)
    want_q, rot_k = rope_ref(q, k, v, positions, cos_sin, neox, dt)
    cache = Cache(Hkv, sum(-(-int(x) // bs) for x in lens) + 3, bs, Hkv, D)
    table = tables(rng, lens, bs, cache.k.shape[0])
    ref.append(rot_k.double().numpy(), cache.k, cache.ks, table, lens, cu)
    ref.append(v.double().numpy(), cache.v, cache.vs, table, lens, cu)
    d = qkv.to(DEV)
    dq = d[:, :Hq]
    q_out = dq if in_place else torch.full((T, Hq, D), 7.0, dtype=DT[dt], device=DEV)
    before = q_out.clone()
    got = rope_append_kv_fp8(dq, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], dev(positions), dev(cos_sin),
                             *cache.dev, dev(table), dev(lens, torch.int32), dev(cu, torch.int64),
                             neox=neox, q_out=q_out)
    cache.check(f"{geom}")
    lo, hi = int(cu[0]), int(cu[-1])
    np.testing.assert_array_equal(bits(got)[lo:hi], bits(want_q)[lo:hi])
    np.testing.assert_array_equal(bits(got)[:lo], bits(before)[:lo])
    np.testing.assert_array_equal(bits(got)[hi:], bits(before)[hi:])
    assert torch.equal(d[:, Hq:], qkv.to(DEV)[:, Hq:])  # k and v are only read


def test_rope_append_bad_positions_write_nothing():
    gen = torch.Generator().manual_seed(9)
    Hq, Hkv, D, bs, dt = 4, 2, 64, 16, "bf16"
    T = 40
    qkv = rows_of(gen, T, Hq + 2 * Hkv, D, dt)
    positions = np.arange(T, dtype=np.int32)
    positions[[3, 20]] = [64, -1]
    live = (positions >= 0) & (positions < 64)
    cos_sin = workloads.rope_cos_sin(64, 64, 10000.0).numpy()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    want_q, rot_k = rope_ref(q, k, v, np.clip(positions, 0, 63), cos_sin, True, dt)
    cache = Cache(8, 4, bs, Hkv, D)
    table, lens, cu = np.array([[1, 3, 0]], np.int32), np.array([T]), np.array([0, T])
    ref.append(rot_k.double().numpy(), cache.k, cache.ks, table, lens, cu, live)
    ref.append(v.double().numpy(), cache.v, cache.vs, table, lens, cu, live)
    d = qkv.to(DEV)
    q_out = torch.full((T, Hq, D), 3.0, dtype=DT[dt], device=DEV)
    err = torch.zeros(2, dtype=torch.int32, device=DEV)
    rope_append_kv_fp8(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], dev(positions), dev(cos_sin),
                       *cache.dev, dev(table), dev(lens, torch.int32), dev(cu, torch.int64),
                       q_out=q_out, err=err)
    cache.check()
    np.testing.assert_array_equal(bits(q_out)[live], bits(want_q)[live])
    assert (q_out[torch.from_numpy(~live).to(DEV)] == 3.0).all()
    assert err.tolist()[0] == 4 and err.tolist()[1] in (3, 20)


# ------------------------------------ read-back ------------------------------------

@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("geom", [(1, 64, 16), (8, 128, 16), (3, 128, 32), (5, 64, 64), (8, 128, 64)])
def test_gather(out, geom):
    Hkv, D, bs = geom
    rng = np.random.default_rng(D + bs)
    lens = np.array([0, 1, bs - 1, bs, bs + 1, 333, 0, 70])
    cache = Cache(D, sum(-(-int(x) // bs) for x in lens) + 2, bs, Hkv, D)
    table = tables(rng, lens, bs, cache.k.shape[0])
    k, v = gather_kv_fp8(*cache.dev, dev(table), dev(lens, torch.int32), dtype=out)
    for got, c, s in ((k, cache.k, cache.ks), (v, cache.v, cache.vs)):
        want = np.concatenate(ref.gather(c, s, table, lens))
        # one rounding of an exact product: torch's cast of the same float64 value (no double
        # rounding: the product has 4 significant bits)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(out))
    cache.check("the cache is only read")


def test_gather_into_given_rows():
    """Sequences in their own rows of a larger buffer: gaps stay, rows and lengths out of range
    are flagged and skipped, a bad block id too."""
    rng = np.random.default_rng(1)
    Hkv, D, bs = 2, 64, 16
    lens = np.array([20, 40, 33])
    cache = Cache(5, 12, bs, Hkv, D)
    table = tables(rng, lens, bs, 12)
    cu = np.array([50, 2, 100])
    k, v = (torch.full((140, Hkv, D), 9.0, device=DEV) for _ in range(2))
    args = (dev(lens, torch.int32),)
    err = torch.zeros(2, dtype=torch.int32, device=DEV)
    gather_kv_fp8(*cache.dev, dev(table), *args, cu_rows=dev(cu, torch.int64), max_len=40, k_out=k, v_out=v, err=err)
    want = np.full((140, Hkv, D), 9.0)
    for b, x in enumerate(ref.gather(cache.k, cache.ks, table, lens)):
        want[cu[b]:cu[b] + lens[b]] = x
    np.testing.assert_array_equal(k.double().cpu().numpy(), want)
    assert err.tolist() == [0, 0]
    # the third sequence's last block leaves the buffer; nothing else changes
    k.fill_(9.0)
    gather_kv_fp8(*cache.dev, dev(table), *args, cu_rows=dev(cu, torch.int64), max_len=40,
                  k_out=k[:132], v_out=v[:132], err=err)
    want[132:] = 9.0
    np.testing.assert_array_equal(k.double().cpu().numpy(), want)
    assert err.tolist() == [2, 2]
    err.zero_()
    bad = table.copy()
    bad[1, 1] = 12
    k.fill_(9.0)
    gather_kv_fp8(*cache.dev, dev(bad), *args, cu_rows=dev(cu, torch.int64), max_len=40, k_out=k,
                  v_out=v, err=err)
    assert err.tolist() == [2, 1]
    assert (k[2 + 16:2 + 32] == 9.0).all() and not (k[2 + 32:2 + 40] == 9.0).all()
    err.zero_()
    gather_kv_fp8(*cache.dev, dev(table), *args, cu_rows=dev(cu, torch.int64), max_len=39, k_out=k,
                  v_out=v, err=err)
    assert err.tolist() == [1, 1]


# ------------------------------------ as used ------------------------------------

def test_nothing_to_do_and_broadcast_rows():
    """No sequences, no rows, sequences without new rows: the cache stays as it is. Rows that
    overlap (a broadcast view) are refused."""
    cache = Cache(14, 6, 16, 2, 64)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64, device=DEV)
    none = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    append_kv_fp8(k, k, *cache.dev, none, i32()[:0], i64(0))
    append_kv_fp8(one, one, *cache.dev, none, i32()[:0], i64(0))
    append_kv_fp8(k, k, *cache.dev, i32(0, 1).view(2, 1), i32(7, 16), i64(0, 0, 0))
    append_kv_fp8(one, one, *cache.dev, i32(0, 1).view(2, 1), i32(7, 16), i64(0, 0, 0))
    append_kv_fp8(one, one, *cache.dev, i32(0, 1).view(2, 1), i32(7, 16), i64(1, 1, 1))
    cache.check()
    got = gather_kv_fp8(*cache.dev, none, i32()[:0])
    assert got[0].shape == (0, 2, 64)
    got = gather_kv_fp8(*cache.dev, i32(0, 1).view(2, 1), i32(0, 0))
    assert got[0].shape == (0, 2, 64)
    with pytest.raises(ValueError, match="overlap"):
        append_kv_fp8(one.expand(3, 2, 64), one.expand(3, 2, 64), *cache.dev, i32(0).view(1, 1), i32(3), i64(0, 3))
    with pytest.raises(ValueError):
        append_kv_fp8(one.transpose(1, 2), one.transpose(1, 2), *cache.dev, i32(0).view(1, 1), i32(1), i64(0, 1))
    wide = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        rope_kv_write(one.expand(3, 2, 64), one.expand(3, 2, 64), one.expand(3, 2, 64), i32(0, 1, 2), i64(0, 1, 2),
                      torch.zeros(4, 64, device=DEV), wide, wide.clone())
    cache.check()


def test_two_streams_append_to_their_own_sequences():
    """Calls on two streams at once, each for sequences of its own, in one cache."""
    gen = torch.Generator().manual_seed(15)
    Hkv, D, bs, n = 8, 128, 16, 2000
    cache = Cache(15, 2 * 125 + 1, bs, Hkv, D)
    order = np.random.default_rng(15).permutation(250).astype(np.int32)
    x = rows_of(gen, 2 * n, 2 * Hkv, D, "bf16")
    parts = []
    for i in range(2):
        rows, table = x[i * n:(i + 1) * n], order[i * 125:(i + 1) * 125][None]
        ref.append(rows[:, :Hkv].double().numpy(), cache.k, cache.ks, table, [n], [0, n])
        ref.append(rows[:, Hkv:].double().numpy(), cache.v, cache.vs, table, [n], [0, n])
        parts.append((rows.to(DEV), dev(table), dev(np.array([n]), torch.int32), dev(np.array([0, n]), torch.int64)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):  # the same rows again: blocks that start anew hold the same
        for (rows, table, lens, cu), s in zip(parts, streams):
            append_kv_fp8(rows[:, :Hkv], rows[:, Hkv:], *cache.dev, table, lens, cu, stream=s)
    cache.check()


def test_calls_are_captured_and_replayed_on_another_stream():
    """A decode step's append in a CUDA graph on a side stream: every replay appends the next
    token from the tensors it was captured with."""
    rng = np.random.default_rng(11)
    B, Hkv, D, bs, steps = 4, 2, 64, 16, 20
    cache = Cache(6, 16, bs, Hkv, D)
    table = rng.permutation(16).reshape(4, 4)[:, :].astype(np.int32)
    lens = np.array([3, 16, 0, 30])
    x = torch.from_numpy(rng.standard_normal((steps, B, 2 * Hkv, D)).astype(np.float32) *
                         np.exp2(rng.integers(-4, 4, (steps, 1, 1, 1))).astype(np.float32)).to(torch.bfloat16)
    buf = torch.zeros(B, 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    dlens, dt, cu = dev(lens, torch.int32), dev(table), torch.arange(B + 1, device=DEV)
    xs = x.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dlens.add_(1)
        append_kv_fp8(buf[:, :Hkv], buf[:, Hkv:], *cache.dev, dt, dlens, cu)
    with torch.cuda.stream(side):
        for t in range(steps):
            buf.copy_(xs[t])
            graph.replay()
    side.synchronize()
    for t in range(steps):
        lens = lens + 1
        ref.append(x[t, :, :Hkv].double().numpy(), cache.k, cache.ks, table, lens, np.arange(B + 1))
        ref.append(x[t, :, Hkv:].double().numpy(), cache.v, cache.vs, table, lens, np.arange(B + 1))
    cache.check()


def test_shared_block_is_copied_before_an_append():
    """Two sequences share a half-filled block: the block and its scales are copied for one of
    them (copy_blocks for the bytes), then both append; neither sees the other's token."""
    gen = torch.Generator().manual_seed(12)
    Hkv, D, bs = 4, 64, 16
    cache = Cache(9, 4, bs, Hkv, D)
    kc, vc, ks, vs = cache.dev
    copy_blocks(kc, vc, torch.tensor([[1, 3]], device=DEV))
    copy_blocks(ks.view(4, 1, 1, Hkv), vs.view(4, 1, 1, Hkv), torch.tensor([[1, 3]], device=DEV))
    for a in (cache.k, cache.v, cache.ks, cache.vs):
        a[3] = a[1]
    cache.check("copied")
    table, lens, cu = np.array([[1], [3]], np.int32), np.array([8, 8]), np.array([0, 1, 2])
    x = rows_of(gen, 2, 2 * Hkv, D, "bf16", spread=3.0)
    ref.append(x[:, :Hkv].double().numpy(), cache.k, cache.ks, table, lens, cu)
    ref.append(x[:, Hkv:].double().numpy(), cache.v, cache.vs, table, lens, cu)
    xd = x.to(DEV)
    append_kv_fp8(xd[:, :Hkv], xd[:, Hkv:], kc, vc, ks, vs, dev(table), dev(lens, torch.int32),
                  dev(cu, torch.int64))
    cache.check()
