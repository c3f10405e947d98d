"""Plain 64-bit decode attention with capped, biased and windowed scores, and how far a kernel
may be from it: shared by the tests of run(softcap, alibi_slopes, window) and of
run_shared_prefix.

The bound per output element, with w the exact weights and out the exact result:
  - half a step of the output type at out;
  - the weights' own rounding to 16 bits, relative 2^-8 (bf16) or 2^-11 (fp16), whose
    denominator adds the rounded weights: sum_t w_t u |v_t - out|;
  - a score is off by at most ds_t: the product in fp32 sums D terms (D + 2 roundings of
    2^-24 of sum |q k|), scale and cap add three more of the score, the tanh is formed as
    1 - 2 / (1 + e^2y) with an error of 2^-21 of the cap (for caps up to 128; of 2^-20 of the
    score above), the bias rounds once, the difference from the maximum once more of either;
    exp by the special-function unit 2^-21 relative: sum_t w_t (2 ds_t + 2^-21) |v_t - out|,
    the factor 2 for the next order of e^ds;
  - products with V and sums in fp32, over up to L terms in chunks: 2^-16 sum_t w_t |v_t|.
"""
import math

import torch


def reference(q, k_cache, v_cache, table, lens, scale, softcap=0.0, slopes=None, window=0):
    """(out, tol) in float64 on the CPU; out[b] of an empty context is 0."""
    B, Hq, D = q.shape
    _, bs, Hkv, _ = k_cache.shape
    G = Hq // Hkv
    q, kc, vc = q.cpu().double(), k_cache.cpu(), v_cache.cpu()
    table, lens = table.cpu().long(), lens.cpu().tolist()
    u = torch.finfo(k_cache.dtype).eps / 2
    out, tol = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    for b, L in enumerate(lens):
        L = max(0, min(L, table.shape[1] * bs))
        lo = max(0, L - window) if window else 0
        if L == 0:
            continue
        at = torch.arange(lo, L)
        ids = table[b, at // bs]
        ok = (ids >= 0) & (ids < kc.shape[0])
        ids = torch.where(ok, ids, 0)
        k = torch.where(ok[:, None, None], kc[ids, at % bs].double(), 0.0)
        v = torch.where(ok[:, None, None], vc[ids, at % bs].double(), 0.0)
        for h in range(Hkv):
            qq = q[b, h * G:(h + 1) * G]
            s = qq @ k[:, h].T * scale
            mag = qq.abs() @ k[:, h].abs().T * abs(scale)
            ds = (D + 2) * 2.0 ** -24 * mag + 3 * 2.0 ** -24 * s.abs()
            if softcap:
                ds += 2.0 ** -21 * softcap if softcap <= 128 else 2.0 ** -20 * s.abs()
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                far = slopes[h * G:(h + 1) * G].cpu().double()[:, None] * (at - (L - 1)).double()
                ds += 2.0 ** -23 * (far.abs() + s.abs())
                s = s + far
            ds += 2.0 ** -23 * (s.abs() + s.amax(1, keepdim=True).abs())
            w = torch.softmax(s, 1)
            o = w @ v[:, h]
            out[b, h * G:(h + 1) * G] = o
            spread = torch.stack([(w[g] * (u + 2 * ds[g] + 2.0 ** -21)) @ (v[:, h] - o[g]).abs()
                                  for g in range(G)])
            tol[b, h * G:(h + 1) * G] = spread + 2.0 ** -16 * (w @ v[:, h].abs())
    step = torch.exp2(torch.floor(torch.log2(out.abs().clamp(min=2.0 ** -24)))) * u
    return out, tol + step * (1 + 1e-9) + 2.0 ** -25


def check(got, want, tol, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() - tol
    worst = int(bad.argmax())
    assert bad.max() <= 0, (f"{what}: {int((bad > 0).sum())} of {bad.numel()} off, worst at {worst}: "
                            f"{got.flatten()[worst]} for {want.flatten()[worst]} +- {tol.flatten()[worst]}")


def make(batch_lens, hq, hkv, d, bs, dtype, groups=(), seed=0, device="cuda", extra=3, spread=1.0):
    """q, caches, table, lens. groups: (first, last, prefix tokens): sequences first .. last - 1 share
    the blocks of their first prefix tokens."""
    gen = torch.Generator().manual_seed(seed)
    B = len(batch_lens)
    pages = [-(-max(0, n) // bs) for n in batch_lens]
    shared = [0] * B
    for a, z, n in groups:
        for b in range(a, z):
            shared[b] = n // bs
    total = sum(n // bs for _, _, n in groups) + sum(max(0, p - s) for p, s in zip(pages, shared)) + extra
    ids = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((B, max(1, max(pages, default=1))), -7, dtype=torch.int32)
    at = 0
    for a, z, n in groups:
        m = n // bs
        for b in range(a, z):
            table[b, :min(m, table.shape[1])] = ids[at:at + min(m, table.shape[1])]
        at += m
    for b in range(B):
        m = max(0, pages[b] - shared[b])
        table[b, shared[b]:shared[b] + m] = ids[at:at + m]
        at += m
    q = (spread * torch.randn(B, hq, d, generator=gen)).to(dtype)
    k = torch.randn(total, bs, hkv, d, generator=gen).to(dtype)
    v = (torch.randn(total, bs, hkv, d, generator=gen) + 0.5).to(dtype)
    lens = torch.tensor(list(batch_lens), dtype=torch.int32)
    return [t.to(device) for t in (q, k, v, table, lens)]


def poison(k, v, table, lens, window=0):
    """NaN and infinities in every row of the caches that no sequence may see (in place)."""
    nb, bs = k.shape[:2]
    seen = torch.zeros(nb, bs, dtype=torch.bool)
    t, ln = table.cpu().long(), lens.cpu().tolist()
    for b, L in enumerate(ln):
        at = torch.arange(max(0, L - window) if window else 0, max(0, L))
        seen[t[b, at // bs], at % bs] = True
    seen = seen.to(k.device)
    k[~seen] = math.nan
    v[~seen] = math.inf
