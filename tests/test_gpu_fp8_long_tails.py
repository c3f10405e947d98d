"""Decode attention over FP8 caches where one token dominates and the rest of a
long context holds little weight each, as behind the first token of most
prompts: what the small weights add up to counts.

Tolerance, from the kernel's arithmetic. A weight P' (relative to the largest of
its row, 1) is three E4M3 terms, each with an exponent range of its own, in all
off by at most max(2^-13 P', 2^-28). The sums: a thread adds up to L / 128 weights
and the accumulators take L / 128 folds of 128-token products, each addition off by
2^-24 of the running value; at L = 131072 that is 2^-14 for either. A logit is off by
at most delta = scale * (Q sum |q_i k_i| + 2^-17 max |q| sum |k_i|) + 2^-20 (|s| + 64)
with Q = 2 D 2^-24, plus 2^-12 for fp16 queries of more than bf16's 8 bits (three E4M3
terms; the two terms that the per-head call takes hold 8), which moves a weight by at
most exp(2 delta). So
  |out - exact| <= (2^-12 + 4 delta) sum w |v| + 2^-28 max(w vs) sum_t |v8_t| + half a
step of the output type,
which stays below the flat 2e-3 of fp32 output in every case here.
"""
import numpy as np
import pytest
import torch

import fp8_cache_ref as ref
from paged_gqa_decode_attention_gb300 import PagedDecodeAttention

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda", torch.cuda.current_device())
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
SHARES = (0.5, 0.8, 0.95, 0.99)


class Tail:
    """One sequence for each of SHARES, all over the same pages but for the first, whose first
    token holds about that share of the weight. The other tokens' logits deviate by 0.5; values
    have mean 1 and deviation 1, the dominant token's are 0."""

    def __init__(self, G, Hkv, D, bs, L, dt, q_bits8=False):
        rng = np.random.default_rng(L + 17 * G + D)
        pages = L // bs
        assert pages * bs == L
        nb, B = pages - 1 + len(SHARES), len(SHARES)
        self.G, self.Hkv, self.D, self.bs, self.L, self.dt = G, Hkv, D, bs, L, dt
        self.q_terms = 3 if dt == "fp16" and not q_bits8 else 2
        q = np.abs(rng.standard_normal((1, G * Hkv, D))) + 0.5
        self.q = torch.from_numpy(np.repeat(q, B, 0)).to(torch.bfloat16 if q_bits8 else DT[dt]).to(DT[dt])
        self.scale = float(np.float32(D ** -0.5))
        # logits: a byte value of 1 in every dimension is worth `unit`; 448 of them the largest gap
        total, norm = q.sum(-1).mean(), np.sqrt((q ** 2).sum(-1)).mean()
        gap = [np.log(s / (1 - s) * (L - 1)) for s in SHARES]
        unit = max(gap) / 440.0
        self.ks = unit / (self.scale * total)
        k8 = np.empty((nb, bs, Hkv, D), np.uint8)
        v8 = np.empty_like(k8)
        for i in range(0, nb, 256):
            shape = k8[i:i + 256].shape
            k8[i:i + 256] = ref.encode(rng.standard_normal(shape) * (0.5 * total / (norm * unit)))
            v8[i:i + 256] = ref.encode(rng.standard_normal(shape) * 60 + 60)
        order = rng.permutation(nb).astype(np.int32)
        self.table = np.empty((B, pages), np.int32)
        self.table[:, 1:] = order[None, B:]
        self.table[:, 0] = order[:B]
        for b, g in enumerate(gap):
            k8[order[b], 0] = ref.encode(np.full((Hkv, D), g / unit))
            v8[order[b], 0] = 0
        self.k8, self.v8, self.nb = k8, v8, nb

    def want(self, ks, vs):
        """(exact, tolerance) for per-head scales ks, vs [Hkv]."""
        B, Hq, D = self.q.shape
        out, tol = np.zeros(self.q.shape), np.zeros(self.q.shape)
        Q = 2 * D * 2.0 ** -24 + (2.0 ** -12 if self.q_terms == 3 else 0.0)
        for h in range(self.Hkv):
            for b in range(B):
                k = ref.decode(self.k8[self.table[b], :, h]).reshape(self.L, D)
                v = ref.decode(self.v8[self.table[b], :, h]).reshape(self.L, D)
                heads = slice(h * self.G, (h + 1) * self.G)
                q = self.q[b, heads].double().numpy()
                s = self.scale * float(ks[h]) * (q @ k.T)
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                absk = np.abs(k)
                delta = self.scale * float(ks[h]) * (
                    Q * (np.abs(q) @ absk.T) + 2.0 ** -17 * np.abs(q).max(1)[:, None] * absk.sum(1)[None]
                ) + 2.0 ** -20 * (np.abs(s) + 64)
                absv = np.abs(v)
                out[b, heads] = float(vs[h]) * (w @ v)
                tol[b, heads] = float(vs[h]) * (
                    (2.0 ** -12 + 4 * delta.max(1))[:, None] * (w @ absv) +
                    2.0 ** -28 * w.max(1)[:, None] * absv.sum(0)[None])
        return out, tol

    def args(self):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
        fp8 = torch.float8_e4m3fn
        lens = torch.full((len(SHARES),), self.L, dtype=torch.int32, device=DEV)
        return self.q.to(DEV), d(self.k8).view(fp8), d(self.v8).view(fp8), d(self.table), lens, self.scale

    def attn(self):
        return PagedDecodeAttention(self.G * self.Hkv, self.Hkv, self.D, self.bs, DT[self.dt],
                                    max_batch=len(SHARES), max_blocks_per_seq=self.L // self.bs, kv_fp8=True)


def check(got, want, what):
    out, tol = want
    g = got.double().cpu().numpy()
    if got.dtype == torch.float32:
        assert np.abs(g - out).max() < 2e-3, f"{what}: {np.abs(g - out).max():.3e}"
    tol = tol + torch.finfo(got.dtype).eps / 2 * np.abs(out) + 2.0 ** -24
    ratio = np.abs(g - out) / tol
    i = np.unravel_index(np.argmax(ratio), ratio.shape)
    assert ratio[i] <= 1, f"{what}: {i} got {g[i]!r} want {out[i]!r} tolerance {tol[i]:.3e}"


CASES = [(1, 1, 128, 16, 32768, "bf16"), (4, 2, 128, 16, 8192, "bf16"), (4, 1, 128, 16, 131072, "bf16"),
         (4, 1, 64, 32, 32768, "fp16"), (8, 1, 128, 32, 32768, "fp16"), (8, 1, 128, 16, 131072, "bf16"),
         (7, 2, 64, 64, 8192, "bf16"), (7, 1, 64, 64, 32768, "bf16"), (16, 1, 128, 16, 32768, "bf16"),
         (16, 1, 64, 32, 131072, "fp16")]


@pytest.mark.parametrize("G,Hkv,D,bs,L,dt", CASES)
def test_block_scaled_long_tail_behind_a_dominant_token(G, Hkv, D, bs, L, dt):
    t = Tail(G, Hkv, D, bs, L, dt)
    ks, vs = np.full(Hkv, t.ks, np.float32), np.full(Hkv, 1 / 64, np.float32)
    want = t.want(ks, vs)
    scales = dict(k_scale=torch.from_numpy(np.tile(ks, (t.nb, 1))).to(DEV),
                  v_scale=torch.from_numpy(np.tile(vs, (t.nb, 1))).to(DEV))
    args = t.args()
    with t.attn() as attn:
        for s in (1, 0, 3):
            check(attn.run(*args, **scales, num_splits=s, out_dtype=torch.float32), want, f"splits {s}")
        check(attn.run(*args, **scales, num_splits=1), want, dt)
        assert attn.check_device_error() == (0, 0)


@pytest.mark.parametrize("G,Hkv,D,bs,L,dt", CASES)
def test_per_head_scales_long_tail_behind_a_dominant_token(G, Hkv, D, bs, L, dt):
    t = Tail(G, Hkv, D, bs, L, dt, q_bits8=True)
    ks, vs = np.full(Hkv, t.ks, np.float32), np.full(Hkv, 1 / 64, np.float32)
    want = t.want(ks, vs)
    scales = dict(k_scale=torch.from_numpy(ks).to(DEV), v_scale=torch.from_numpy(vs).to(DEV))
    args = t.args()
    with t.attn() as attn:
        for s in (1, 0, 3):
            check(attn.run(*args, **scales, num_splits=s, out_dtype=torch.float32), want, f"splits {s}")
        check(attn.run(*args, **scales, num_splits=1), want, dt)
        assert attn.check_device_error() == (0, 0)
