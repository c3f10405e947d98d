"""Inputs of decode attention whose output shows how finely the weights enter the product with V,
the exact output, and how far a kernel whose weights are the sum of two 16-bit terms may be from it.

Every token belongs to one of eight classes, and any eight tokens from a multiple of eight on have
one of each. Scores depend on the class only, and each dim of V is A for one class, -B for another
and 0 for the rest, with B such that the two nearly cancel: the output is some 2^-5 or less of
sum_t w_t |v_t|, so that its own rounding hides little of what the weights lose.

The bound per element, S = sum_t w_t |v_t|:
  - half a step of the output type at out;
  - two 16-bit terms: S times 2^-16 (bf16) or 2^-22 (fp16; no weight here is below 2^-17 of the
    largest, from where on the second term has fewer bits);
  - a score is off by at most ds: q . k is one exact product, the scale, the difference from the
    maximum and the bias round by 2^-24 of what they work on (six roundings counted), a cap adds
    2^-21 of itself; the exponential by the special-function unit 2^-21: S (2 ds + 2^-21);
  - products and sums in fp32 over up to 2^12 tokens: 2^-16 S, as for plain decode attention.
"""
import torch

from row_attn_ref import make

CLASSES = 8
SCORES = (0.0, -0.3125, -0.71875, -1.046875, -1.453125, -1.859375, -2.28125, -2.671875)  # of q . k, before the scale


def two_terms(dtype):
    return 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22


def make_terms(lens, hq, hkv, d, bs, dtype, groups=(), seed=0, scale=1.0, device="cpu"):
    """As row_attn_ref.make, with the values above; `scale` is what the call will get."""
    q, k, v, table, ln = make(lens, hq, hkv, d, bs, dtype, groups, seed=seed, device="cpu")
    gen = torch.Generator().manual_seed(seed + 1000)
    width = table.shape[1] * bs
    order = torch.cat([torch.randperm(CLASSES, generator=gen) for _ in range(-(-width // CLASSES))])[:width]
    sign = 1.0 if scale >= 0 else -1.0
    value = torch.tensor(SCORES) * sign
    w = torch.exp(abs(scale) * torch.tensor(SCORES, dtype=torch.float64))
    pairs = [(i, j) for i in range(CLASSES) for j in range(CLASSES) if i < j]
    rows = torch.zeros(CLASSES, d, dtype=torch.float64)  # V of each class
    for x in range(d):
        i, j = pairs[x % len(pairs)]
        a = 1.0 + torch.rand(1, generator=gen).item()
        rows[i, x], rows[j, x] = a, -a * w[i] / w[j]
    rows = rows.to(dtype)
    q[..., 0] = 1.0
    k.zero_()
    v.zero_()
    for b, n in enumerate(lens):
        at = torch.arange(max(0, n))
        ids = table[b, at // bs].long()
        k[ids, at % bs, :, 0] = value[order[at]].to(dtype)[:, None]
        v[ids, at % bs] = rows[order[at]][:, None]
    return [t.to(device) for t in (q, k, v, table, ln)]


def reference(q, k, v, table, lens, scale, softcap=0.0, slopes=None, window=0, weights=None):
    """(out, tol) in float64 on the CPU. weights(p) -> (weights, sum): what a kernel makes of the
    weights relative to the largest one; None: exact."""
    q, k, v, table = q.cpu().double(), k.cpu(), v.cpu(), table.cpu().long()
    B, hq, d = q.shape
    bs, hkv = k.shape[1], k.shape[2]
    g, u = hq // hkv, torch.finfo(k.dtype).eps / 2
    out, tol = torch.zeros(B, hq, d, dtype=torch.float64), torch.zeros(B, hq, d, dtype=torch.float64)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        at = torch.arange(max(0, n - window) if window else 0, n)
        kk, vv = (x[table[b, at // bs], at % bs].double() for x in (k, v))
        s = torch.einsum("hgd,thd->hgt", q[b].view(hkv, g, d), kk) * scale
        ds = 6 * 2.0 ** -24 * s.abs().max()
        if softcap:
            ds += 2.0 ** -21 * softcap
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            far = slopes.cpu().double().view(hkv, g, 1) * (at - (n - 1)).double()
            # only what is near the last token has weight; a far score's error is of its own size
            ds = ds + 6 * 2.0 ** -24 * far.abs()
            s = s + far
        p = torch.exp(s - s.amax(-1, keepdim=True))
        total = p.sum(-1, keepdim=True)
        share = p / total
        used, by = (p, total) if weights is None else weights(p)
        out[b] = (torch.einsum("hgt,thd->hgd", used, vv) / by).reshape(hq, d)
        off = two_terms(k.dtype) + 2 * ds + 2.0 ** -21 + 2.0 ** -16
        tol[b] = torch.einsum("hgt,thd->hgd", share * off, vv.abs()).reshape(hq, d)
    step = torch.exp2(torch.floor(torch.log2(out.abs().clamp(min=2.0 ** -14)))) * u
    return out, tol + step * (1 + 1e-9)


# (own tokens of each sequence, shared tokens, Hq, Hkv, D, block size, type)
SHARED = [
    ([40] * 17, 640, 16, 2, 128, 16, torch.bfloat16),          # 136 rows: one wide tile
    ([33, 200] * 20, 1024, 16, 2, 64, 32, torch.bfloat16),     # a wide tile and one of 64 rows
    ([24] * 40, 900, 8, 1, 128, 16, torch.float16),
    ([56] * 70, 512, 4, 1, 64, 16, torch.float16),
    ([50] * 16, 640, 16, 2, 128, 16, torch.bfloat16),          # 128 rows: not wide
]
# (lengths, Hq, Hkv, D, block size, type, cap, window)
OWN = [
    ([700, 200, 1333], 8, 2, 128, 16, torch.bfloat16, 0.0, 640),
    ([900, 160], 14, 2, 64, 16, torch.bfloat16, 2.0, 0),
    ([1500, 257], 16, 1, 64, 32, torch.float16, 2.0, 1024),
    ([333] * 5, 4, 4, 128, 16, torch.float16, 0.0, 300),
]
