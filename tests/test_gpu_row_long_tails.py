"""run_shared_prefix and run(softcap, window) where one token dominates and the rest of a long
context holds little weight each: the token in a sequence's own part or in the shared one, tiles of
128 rows and of more.

Tolerance, from the kernel's arithmetic: a weight is two 16-bit terms, off by at most 2^-16 of it in
bf16 or, in fp16 at p * 2^14, by 2^-22 of it or 2^-39 of the largest, whichever is more. Sums: up to 1024
additions of 2^-24 each in a thread and in the accumulators. A score is off by
delta = 2 D 2^-24 scale sum |q_i k_i| + 2^-20 (|s| + 64) + 2^-21 cap, which moves a weight by at most
exp(2 delta). So
  |out - exact| <= (2^-12 + 4 delta) sum w |v| + 2^-39 max(w) sum_t |v_t| + half a step."""
import numpy as np
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
SHARES = (0.5, 0.95, 0.99, 0.999, 0.9999)


def expected(q, kk, vv, scale, cap):
    D = q.shape[-1]
    kk, vv, q = kk.double(), vv.double(), q.double()
    s = scale * (q @ kk.T)
    delta = 2 * D * 2.0 ** -24 * scale * (q.abs() @ kk.abs().T) + 2.0 ** -20 * (s.abs() + 64) + 2.0 ** -21 * cap
    if cap:
        s = cap * torch.tanh(s / cap)
    w = torch.softmax(s, -1)
    tol = (2.0 ** -12 + 4 * delta.amax(-1))[:, None] * (w @ vv.abs())
    return w @ vv, tol + 2.0 ** -39 * w.amax(-1)[:, None] * vv.abs().sum(0)[None]


def inputs(G, D, bs, L, dt, tops):
    """q [G, D], K and V of `tops` first blocks (a dominant token each) and of L tokens more."""
    gen = torch.Generator(device="cuda").manual_seed(G * D + bs)
    nb = L // bs + len(tops)
    scale = float(np.float32(D ** -0.5))
    q = torch.randn(G, D, generator=gen, device="cuda").abs().add(0.5).to(dt)
    k = torch.randn(nb, bs, 1, D, generator=gen, device="cuda") * (0.5 / (scale * float(q.float().norm(dim=-1).mean())))
    v = torch.randn(nb, bs, 1, D, generator=gen, device="cuda") * 2 + 4
    for b, share in enumerate(tops):
        k[b, 0] = np.log(share / (1 - share) * L) / (scale * float(q.float().sum(-1).mean()))
        v[b, 0] = 0
    return q, k.to(dt), v.to(dt), scale


def compare(out, want, tol, dt, what):
    over = (out.double() - want).abs() - tol - torch.finfo(dt).eps / 2 * want.abs() - 2.0 ** -25
    assert float(over.max()) <= 0, (what, float((out.double() - want).abs().max()))


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("G,D,bs,L", [(4, 128, 16, 131072), (8, 64, 32, 32768), (7, 128, 16, 32768), (1, 64, 16, 8192)])
@pytest.mark.parametrize("cap", [0.0, 60.0])
def test_own_part(dt, G, D, bs, L, cap):
    q, k, v, scale = inputs(G, D, bs, L, dt, SHARES)
    B, n = len(SHARES), L // bs
    table = torch.arange(B, B + n, dtype=torch.int32, device="cuda").repeat(B, 1)
    table = torch.cat([torch.arange(B, dtype=torch.int32, device="cuda")[:, None], table], 1).contiguous()
    ln = torch.full((B,), L + bs, dtype=torch.int32, device="cuda")
    with PagedDecodeAttention(G, 1, D, bs, dt, max_batch=B, max_blocks_per_seq=n + 1, max_splits=1) as a:
        out = a.run(q.repeat(B, 1, 1), k, v, table, ln, scale, softcap=cap, window=0 if cap else L + bs)
        assert a.check_device_error() == (0, 0)
    for b in range(B):
        kk, vv = (x[table[b].long()].view(-1, D) for x in (k, v))
        compare(out[b], *expected(q, kk, vv, scale, cap), dt, b)


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("G,D,bs,L", [(4, 128, 16, 32768), (8, 64, 32, 16384)])
@pytest.mark.parametrize("rows", [32, 128, 256, 320])
@pytest.mark.parametrize("where", ["own", "shared"])
def test_shared_part(dt, G, D, bs, L, rows, where):
    B, n = rows // G, L // bs
    tops = SHARES if where == "own" else SHARES[-1:]
    q, k, v, scale = inputs(G, D, bs, L, dt, tops)
    shared = torch.arange(len(tops), len(tops) + n, dtype=torch.int32, device="cuda").repeat(B, 1)
    first = (torch.arange(B, dtype=torch.int32, device="cuda") % len(tops))[:, None]
    table = torch.cat([shared, first] if where == "own" else [first, shared], 1).contiguous()
    ln = torch.full((B,), L + bs, dtype=torch.int32, device="cuda")
    cu, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, B], [L if where == "own" else L + bs]))
    with PagedDecodeAttention(G, 1, D, bs, dt, max_batch=B, max_blocks_per_seq=n + 1, max_splits=1) as a:
        out = a.run_shared_prefix(q.repeat(B, 1, 1), k, v, table, ln, cu, pre, scale)
        assert a.check_device_error() == (0, 0)
    for t in range(min(B, len(tops))):
        kk, vv = (x[table[t].long()].view(-1, D) for x in (k, v))
        want, tol = expected(q, kk, vv, scale, 0.0)
        compare(out[t::len(tops)], want, tol, dt, t)
