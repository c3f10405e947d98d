"""GPU parity of decode attention over a block-scaled FP8 cache against plain
64-bit attention, and the cache's calls used together.

Tolerance, from the kernel's arithmetic. A weight P' (relative to the largest
of its row, 1) is split into three E4M3 terms of 256 P', each rounded to
nearest with relative error at most 2^-4 or, among the subnormals, absolute
error at most 2^-10: the split's error is at most max(2^-12 P', 2^-18). A
logit is off by at most delta = scale * (Q * sum |q_i k_i| + 2^-17 max |q|
sum |k_i|) + 2^-20 (|s| + 64) with Q = 2 D 2^-24 for the fp32 sums, plus 2^-12
for fp16 queries (three E4M3 terms), which moves a weight by a factor of at
most exp(2 delta). So
  |out - exact| <= (2^-11 + 4 delta) sum w |v| + sum_t 2^-18 max(w' vs) |v8_t| + half a step of the
output type, w the exact probabilities, w' vs their products with the V scales.
"""
import numpy as np
import pytest
import torch

import fp8_cache_ref as ref
from paged_gqa_decode_attention_gb300 import (PDA_EINVAL, PDAError, PagedDecodeAttention,
                                              append_kv_fp8, gather_kv_fp8, rope_append_kv_fp8,
                                              rope_kv_write, workloads)

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda", torch.cuda.current_device())
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
FP8 = torch.float8_e4m3fn


def expect(q, kc, vc, ks, vs, table, lens, scale, fp16):
    """(exact output, tolerance before the output's own rounding), [B, Hq, D] float64."""
    B, Hq, D = q.shape
    nb, bs, Hkv, _ = kc.shape
    G = Hq // Hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        blk = np.asarray(table[b])[:-(-L // bs)]
        ok = (blk >= 0) & (blk < nb)
        safe = np.where(ok, blk, 0)
        k8 = np.where(ok[:, None, None, None], ref.decode(kc[safe]), 0.0).reshape(-1, Hkv, D)[:L]
        v8 = np.where(ok[:, None, None, None], ref.decode(vc[safe]), 0.0).reshape(-1, Hkv, D)[:L]
        kss = np.repeat(np.where(ok[:, None], ks[safe], 0.0).astype(np.float64), bs, 0)[:L]
        vss = np.repeat(np.where(ok[:, None], vs[safe], 0.0).astype(np.float64), bs, 0)[:L]
        for h in range(Hkv):
            k, v = k8[:, h] * kss[:, h, None], v8[:, h] * vss[:, h, None]
            qq = q[b, h * G:(h + 1) * G]
            s = scale * (qq @ k.T)                                       # [G, L]
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[b, h * G:(h + 1) * G] = w @ v
            qk = np.abs(qq) @ np.abs(k).T
            Q = 2 * D * 2.0 ** -24 + (2.0 ** -12 if fp16 else 0.0)
            delta = abs(scale) * (Q * qk + 2.0 ** -17 * np.abs(qq).max(1)[:, None] *
                                  np.abs(k).sum(1)[None]) + 2.0 ** -20 * (np.abs(s) + 64)
            # weights that do not matter do not set the bound
            delta = np.where(w > 2.0 ** -40, delta, 0).max(1)
            top = (w * vss[:, h][None]).max(1)
            tol[b, h * G:(h + 1) * G] = ((2.0 ** -11 + 4 * delta)[:, None] * (w @ np.abs(v)) +
                                         2.0 ** -18 * top[:, None] * np.abs(v8[:, h]).sum(0)[None])
    return out, tol


def check(got, want, what=""):
    out, tol = want
    g = got.double().cpu().numpy()
    tol = tol + torch.finfo(got.dtype).eps / 2 * np.abs(out) + 2.0 ** -24  # fp16: subnormal step
    assert np.isfinite(g).all(), what
    bad = np.abs(g - out) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(g - out) / tol), g.shape)
        raise AssertionError(f"{what}: {bad.sum()} beyond tolerance; worst {i}: got {g[i]!r} want "
                             f"{out[i]!r} tolerance {tol[i]:.3e}")


class Problem:
    def __init__(self, seed, G, Hkv, D, bs, lens, dt="bf16", pow2=True, spread=5, extra_blocks=3):
        rng = np.random.default_rng(seed)
        self.lens = np.array(lens)
        pages = [-(-int(x) // bs) for x in lens]
        nb = sum(pages) + extra_blocks
        self.bs, self.D, self.Hkv, self.dt = bs, D, Hkv, dt
        self.kc = ref.encode(rng.standard_normal((nb, bs, Hkv, D)) * 60)
        self.vc = ref.encode(rng.standard_normal((nb, bs, Hkv, D)) * 60)
        self.ks = np.exp2(rng.integers(-8, -4, (nb, Hkv)) if pow2 else rng.uniform(-8, -4, (nb, Hkv))).astype(np.float32)
        self.vs = np.exp2(rng.integers(-spread, spread + 1, (nb, Hkv)) if pow2
                          else rng.uniform(-spread, spread, (nb, Hkv))).astype(np.float32)
        order = rng.permutation(nb)
        self.table = np.full((len(lens), max(1, max(pages))), nb + 1000, np.int32)  # unused: never read
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            # rows past the context and blocks nobody names hold NaN
            if n and int(lens[b]) % bs:
                for c in (self.kc, self.vc):
                    c[order[at + n - 1], int(lens[b]) % bs:] = 0x7F
            at += n
        self.kc[order[at:]] = self.vc[order[at:]] = 0xFF
        self.ks[order[at:]] = self.vs[order[at:]] = np.nan
        self.q = torch.from_numpy(rng.standard_normal((len(lens), G * Hkv, D))).to(DT[dt])
        self.scale = 1.0 / np.sqrt(D)

    def attn(self, **kw):
        return PagedDecodeAttention(self.q.shape[1], self.Hkv, self.D, self.bs, DT[self.dt],
                                    max_batch=len(self.lens), max_blocks_per_seq=self.table.shape[1],
                                    kv_fp8=True, **kw)

    def upload(self):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
        self.dev = (self.q.to(DEV), d(self.kc).view(FP8), d(self.vc).view(FP8), d(self.table),
                    d(self.lens.astype(np.int32)), float(self.scale))
        self.scales = dict(k_scale=d(self.ks), v_scale=d(self.vs))
        return self

    def run(self, attn, **kw):
        out = attn.run(*self.dev, **self.scales, **kw)
        torch.cuda.synchronize()
        assert attn.check_device_error() == (0, 0)
        return out

    def want(self):
        return expect(self.q.double().numpy(), self.kc, self.vc, self.ks, self.vs, self.table, self.lens,
                      float(np.float32(self.scale)), self.dt == "fp16")


def every_way(p, splits=(0, 1, 3, 64)):
    p.upload()
    want = p.want()
    with p.attn() as attn:
        for s in splits:
            check(p.run(attn, num_splits=s), want, f"splits {s}")
        check(p.run(attn, out_dtype=torch.float32), want, "fp32 out")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv,bs", [(1, 8, 16), (2, 3, 32), (3, 2, 64), (4, 8, 16), (4, 1, 64), (5, 2, 16),
                                      (7, 2, 64), (8, 8, 32), (9, 1, 16), (13, 2, 32), (16, 2, 16)])
def test_geometries(dt, D, G, Hkv, bs):
    lens = [1, 0, bs - 1, bs, bs + 1, 127, 128, 129, 700, 1531]
    every_way(Problem(G * 100 + D + bs, G, Hkv, D, bs, lens, dt))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_scales_of_another_quantiser(dt):
    """Scales that are no powers of two."""
    every_way(Problem(5, 4, 2, 128, 16, [900, 17, 2048, 300], dt, pow2=False))


def test_long_contexts_and_cluster_merge():
    every_way(Problem(6, 4, 8, 128, 16, [8192, 8001], "bf16"), splits=(0, 2, 4, 8, 16))
    every_way(Problem(7, 8, 2, 64, 32, [30001], "fp16"), splits=(0, 16, 64))


@pytest.mark.parametrize("B,D,G,Hkv", [(300, 64, 4, 1), (1000, 64, 2, 1), (1024, 64, 8, 1), (1100, 64, 4, 1),
                                       (60, 128, 8, 8)])
def test_many_ragged_sequences(B, D, G, Hkv):
    """More units than CTAs, with and without a directory of the sequences (up to 1024): empty
    contexts, single tokens, a few long ones anywhere in the batch."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 60, B)
    lens[rng.integers(0, B, B // 10)] = 0
    lens[rng.integers(0, B, 9)] = rng.integers(300, 5000, 9)
    every_way(Problem(B, G, Hkv, D, 16, lens), splits=(0, 1, 7))


def test_extreme_block_scales():
    """V scales 2^40 apart, zeros, blocks whose V or K is nothing but zeros, and subnormal scales:
    the probabilities do not suffer from where the large values sit."""
    p = Problem(8, 4, 2, 128, 16, [500, 16, 90, 700], "bf16", spread=20)
    p.vs[p.table[0, 3]], p.vs[p.table[0, 5], 1] = 0.0, 1e-40
    p.ks[p.table[0, 7]], p.ks[p.table[2, 1]] = 0.0, 0.0
    p.vs[p.table[1, 0]] = 0.0            # a sequence whose values are all zero
    p.vs[p.table[2, :6]] = 2.0 ** -70    # all of them below the smallest written scale
    every_way(p)


def test_unlikely_tokens_with_large_values():
    """A block of values 2^30 times larger than the others, seen with probability ~2^-40 and
    ~2^-30: the other blocks' contribution keeps its precision."""
    rng = np.random.default_rng(9)
    for shift in (27.7, 20.8):
        p = Problem(10, 4, 1, 64, 16, [400], "bf16", spread=1)
        q = np.abs(rng.standard_normal(64)) + 0.5
        p.q = torch.from_numpy(np.tile(q, (1, 4, 1))).to(torch.bfloat16)
        p.kc[p.table[0]] = ref.encode(rng.standard_normal((25, 16, 1, 64)) * 2)
        p.kc[p.table[0, 11]] = ref.encode(np.full((16, 1, 64), -448.0))
        norm = float(p.q.double()[0, 0].sum()) * 448
        p.ks[:] = 2.0 ** -8
        p.ks[p.table[0, 11]] = np.float32(shift / norm / p.scale)
        p.vs[p.table[0, 11]] = 2.0 ** 30
        every_way(p, splits=(1, 0))


def test_bad_block_ids_read_zeros():
    p = Problem(11, 4, 2, 128, 16, [100, 60], "bf16")
    p.table[0, 2], p.table[1, 0] = -1, p.kc.shape[0]
    every_way(p)


def test_equal_scales_match_the_per_head_call():
    """One power of two for every block of a head: the same numbers as the per-head scales give."""
    p = Problem(12, 4, 8, 128, 16, [1000, 333, 64], "bf16")
    head = np.exp2(np.arange(8) - 6).astype(np.float32)
    p.ks[:], p.vs[:] = head, head[::-1]
    p.upload()
    with p.attn() as attn:
        a = p.run(attn, out_dtype=torch.float32)
        b = attn.run(*p.dev, k_scale=torch.from_numpy(head).to(DEV),
                     v_scale=torch.from_numpy(head[::-1].copy()).to(DEV), out_dtype=torch.float32)
    want = p.want()
    check(a, want, "block scales")
    check(b, want, "head scales")


def test_scales_of_one_block_and_of_heads_in_two_dimensions():
    """A cache of one block, and per-head scales passed as [1, Hkv], both mean the heads' scales."""
    p = Problem(16, 4, 8, 128, 16, [13], "bf16", extra_blocks=0)
    assert p.ks.shape == (1, 8)
    every_way(p, splits=(0,))
    p = Problem(17, 4, 8, 128, 16, [300, 20], "bf16")
    p.ks[:], p.vs[:] = p.ks[p.table[0, 0]], p.vs[p.table[0, 0]]
    p.upload()
    with p.attn() as attn:
        one = {n: t[int(p.table[0, 0])][None].contiguous() for n, t in p.scales.items()}
        check(attn.run(*p.dev, **one), p.want())


def test_captured_and_replayed_with_a_cache_that_moves_on():
    p = Problem(13, 4, 2, 128, 16, [100, 200], "bf16").upload()
    with p.attn() as attn:
        out = torch.empty_like(p.dev[0])
        attn.run(*p.dev, **p.scales, out=out)
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            attn.run(*p.dev, **p.scales, out=out)
        for step in range(3):
            p.vs[p.table[0, step]] *= 2.0
            p.lens[:] += 5
            p.lens = np.minimum(p.lens, [112, 208])
            p.kc[:] = np.where((p.kc & 0x7F) == 0x7F, 0x30, p.kc)
            p.vc[:] = np.where((p.vc & 0x7F) == 0x7F, 0x30, p.vc)
            p.scales["v_scale"].copy_(torch.from_numpy(p.vs))
            p.dev[1].view(torch.uint8).copy_(torch.from_numpy(p.kc))
            p.dev[2].view(torch.uint8).copy_(torch.from_numpy(p.vc))
            p.dev[4].copy_(torch.from_numpy(p.lens.astype(np.int32)))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            check(out, p.want(), f"replay {step}")


def test_two_handles_on_two_streams_and_an_empty_batch():
    ps = [Problem(18 + i, 4, 2, 128, 16, [900 + i, 33, 400], "bf16").upload() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    attns = [p.attn() for p in ps]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs = [a.run(*p.dev, **p.scales, stream=s) for a, p, s in zip(attns, ps, streams)]
    torch.cuda.synchronize()
    for p, out in zip(ps, outs):
        check(out, p.want())
    q, kc, vc, table, lens, scale = ps[0].dev
    assert attns[0].run(q[:0], kc, vc, table[:0], lens[:0], scale, **ps[0].scales).shape == (0, 8, 128)
    for a in attns:
        a.close()


def test_timed_out_wait_is_reported_and_the_next_run_is_exact(monkeypatch):
    monkeypatch.setenv("PDA_TEST_STALL_RUNS", "1")
    p = Problem(14, 4, 2, 128, 16, [700, 90], "bf16").upload()
    with p.attn() as attn:
        attn.run(*p.dev, **p.scales)
        assert attn.check_device_error()[0] == 3
        check(p.run(attn), p.want())


def test_refusals():
    p = Problem(15, 4, 2, 64, 16, [40], "bf16").upload()
    with p.attn() as attn:
        ks, vs = p.scales["k_scale"], p.scales["v_scale"]
        for a, b in ((ks, None), (None, vs), (ks[:-1].contiguous(), vs), (ks, vs[:, :1].contiguous()), (ks, vs[0])):
            with pytest.raises(ValueError):
                attn.run(*p.dev, k_scale=a, v_scale=b)
        with pytest.raises(ValueError):
            attn.run(*p.dev, k_scale=ks.t().contiguous().t(), v_scale=vs)
        with pytest.raises(ValueError):
            attn.run(*p.dev, k_scale=ks.cpu(), v_scale=vs)
        with pytest.raises(ValueError):
            attn.run(*p.dev, k_scale=ks.half(), v_scale=vs)
        with pytest.raises(ValueError):
            attn.run(p.dev[0][:, :4].contiguous(), *p.dev[1:], k_scale=ks, v_scale=vs)
        with pytest.raises(ValueError):
            attn.run(*p.dev[:4], torch.cat([p.dev[4], p.dev[4]]), p.dev[5], k_scale=ks, v_scale=vs)
        q, kc, vc, table, lens, scale = p.dev
        out = torch.empty_like(q)
        args = lambda k, v, h: (h, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), k, v, table.data_ptr(),
                                lens.data_ptr(), 1, table.shape[1], kc.shape[0], scale, out.data_ptr(), 0, 0, 0, -1)
        call = attn.lib.paged_decode_attn_run_block_scaled
        assert call(*args(None, vs.data_ptr(), attn.handle)) == PDA_EINVAL
        assert call(*args(ks.data_ptr(), vs.data_ptr(), None)) == PDA_EINVAL
        assert call(*args(ks.data_ptr() + 2, vs.data_ptr(), attn.handle)) == PDA_EINVAL
    with PagedDecodeAttention(8, 2, 64, 16, max_batch=1, max_blocks_per_seq=3) as plain:
        k16 = torch.zeros(kc.shape, dtype=torch.bfloat16, device=DEV)
        assert plain.lib.paged_decode_attn_run_block_scaled(
            plain.handle, q.data_ptr(), k16.data_ptr(), k16.data_ptr(), ks.data_ptr(), vs.data_ptr(),
            table.data_ptr(), lens.data_ptr(), 1, table.shape[1], kc.shape[0], scale, out.data_ptr(), 0, 0, 0,
            -1) == PDA_EINVAL
        with pytest.raises((ValueError, PDAError)):
            plain.run(q, k16, k16, table, lens, scale, k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("geom", [(14, 2, 64, 16, "bf16"), (32, 8, 128, 32, "fp16")])
def test_a_generation_as_it_is_served(geom):
    """Prompts are written with rotary positions, then tokens are decoded one by one: each step
    rotates and appends the new rows and attends over the cache; at the end the cache is read
    back. Held against the same steps in 64 bits, and, loosely, against attention over a 16-bit
    cache written by rope_kv_write."""
    Hq, Hkv, D, bs, dt = geom
    G = Hq // Hkv
    rng = np.random.default_rng(D)
    gen = torch.Generator().manual_seed(D)
    prompts, steps = np.array([37, 1, 64]), 20
    B, width = 3, -(-(64 + 20) // bs)
    nb = B * width + 2
    table = rng.permutation(nb)[:B * width].reshape(B, width).astype(np.int32)
    cos_sin = workloads.rope_cos_sin(128, D, 10000.0).to(DEV)
    kc, vc = (torch.zeros(nb, bs, Hkv, D, dtype=FP8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(nb, Hkv, device=DEV) for _ in range(2))
    k16, v16 = (torch.zeros(nb, bs, Hkv, D, dtype=DT[dt], device=DEV) for _ in range(2))
    ref_c = [np.zeros((nb, bs, Hkv, D), np.uint8) for _ in range(2)]
    ref_s = [np.zeros((nb, Hkv), np.float32) for _ in range(2)]
    dtable = torch.from_numpy(table).to(DEV)
    lens = prompts.copy()
    with PagedDecodeAttention(Hq, Hkv, D, bs, DT[dt], max_batch=B, max_blocks_per_seq=width, kv_fp8=True) as attn:
        for step in range(steps + 1):
            new = prompts if step == 0 else np.ones(B, int)
            lens = prompts + step
            cu = np.concatenate([[0], np.cumsum(new)])
            T = int(cu[-1])
            qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen).to(DT[dt]).to(DEV)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            pos = np.concatenate([np.arange(lens[b] - new[b], lens[b]) for b in range(B)]).astype(np.int32)
            dlens = torch.from_numpy(lens.astype(np.int32)).to(DEV)
            q_rot = rope_append_kv_fp8(q, k, v, torch.from_numpy(pos).to(DEV), cos_sin, kc, vc, ks, vs, dtable,
                                       dlens, torch.from_numpy(cu).to(DEV))
            seq = np.repeat(np.arange(B), new)
            slots = table[seq, pos // bs].astype(np.int64) * bs + pos % bs
            want_q = rope_kv_write(q, k, v, torch.from_numpy(pos).to(DEV), torch.from_numpy(slots).to(DEV), cos_sin,
                                   k16, v16)
            assert torch.equal(q_rot, want_q)
            rows = [c.view(-1, Hkv, D)[torch.from_numpy(slots).to(DEV)].double().cpu().numpy() for c in (k16, v16)]
            for x, c, s in zip(rows, ref_c, ref_s):
                ref.append(x, c, s, table, lens, cu)
            if step == 0:
                continue
            out = attn.run(q_rot, kc, vc, dtable, dlens, k_scale=ks, v_scale=vs)
            check(out, expect(q_rot.double().cpu().numpy(), *ref_c, *ref_s, table, lens,
                              float(np.float32(1 / np.sqrt(D))), dt == "fp16"), f"step {step}")
        np.testing.assert_array_equal(kc.view(torch.uint8).cpu().numpy(), ref_c[0])
        np.testing.assert_array_equal(vc.view(torch.uint8).cpu().numpy(), ref_c[1])
        back_k, back_v = gather_kv_fp8(kc, vc, ks, vs, dtable, dlens, dtype=DT[dt])
        exact = [np.concatenate(ref.gather(c, s, table, lens)) for c, s in zip(ref_c, ref_s)]
        np.testing.assert_array_equal(back_k.double().cpu().numpy(), exact[0])
        np.testing.assert_array_equal(back_v.double().cpu().numpy(), exact[1])
        # every stored value is within an E4M3 rounding of the 16-bit one: 2^-4 relative, or half
        # the subnormal step 2^-9 of its block's scale; once more for each requantisation (at
        # most one a doubling of the scale, and only among subnormals)
        full16 = np.concatenate([k16[dtable[b].long()].view(-1, Hkv, D)[:lens[b]].double().cpu().numpy() for b in range(B)])
        scale_rows = np.concatenate([np.repeat(ref_s[0][table[b]], bs, 0)[:lens[b]] for b in range(B)]).astype(np.float64)
        assert (np.abs(exact[0] - full16) <= 2.0 ** -4 * np.abs(full16) + 2.0 ** -9 * scale_rows[:, :, None]).all()
