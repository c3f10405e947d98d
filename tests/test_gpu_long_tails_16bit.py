"""Decode attention over 16-bit caches where one token dominates and the rest of a
long context holds little weight each (both kernels).

Tolerance, from the kernels' arithmetic: the tensor-core kernel takes a weight as two
16-bit terms, off by at most 2^-16 of it (bf16: 2^-9 2^-8, halved by rounding) or, in fp16
at p * 2^14, by 2^-39 of the largest; the CUDA-core kernel takes it in fp32. Sums: up to
1024 additions of 2^-24 each in a thread and in the accumulators. A logit is off by
delta = 2 D 2^-24 scale sum |q_i k_i| + 2^-20 (|s| + 64), which moves a weight by at most
exp(2 delta). So
  |out - exact| <= (2^-12 + 4 delta) sum w |v| + 2^-39 max(w) sum_t |v_t| + half a step."""
import numpy as np
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda", torch.cuda.current_device())
SHARES = (0.5, 0.95, 0.99, 0.999, 0.9999)


@pytest.mark.parametrize("kernel", ["tensor_core", "cuda_core"])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("G,D,bs,L", [(4, 128, 16, 131072), (4, 64, 32, 32768), (8, 128, 16, 32768),
                                      (7, 64, 16, 131072), (1, 128, 32, 8192)])
def test_long_tail_behind_a_dominant_token(kernel, dt, G, D, bs, L, monkeypatch):
    monkeypatch.setenv("PDA_PARTIAL_KERNEL", kernel)
    gen = torch.Generator(device=DEV).manual_seed(G * D + bs)
    B, nb = len(SHARES), L // bs + len(SHARES)
    scale = float(np.float32(D ** -0.5))
    q = torch.randn(1, G, D, generator=gen, device=DEV).abs().add(0.5).to(dt).expand(B, G, D).contiguous()
    k = torch.randn(nb, bs, 1, D, generator=gen, device=DEV) * (0.5 / (scale * float(q.float().norm(dim=-1).mean())))
    v = torch.randn(nb, bs, 1, D, generator=gen, device=DEV) * 2 + 4
    table = torch.arange(nb - L // bs, nb, dtype=torch.int32, device=DEV).repeat(B, 1)
    table[:, 0] = torch.arange(B, device=DEV)  # each share's own first block
    for b, share in enumerate(SHARES):
        k[b, 0] = np.log(share / (1 - share) * (L - 1)) / (scale * float(q.float().sum(-1).mean()))
        v[b, 0] = 0
    k, v = k.to(dt), v.to(dt)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    want, tol = [], []
    for b in range(B):
        kk, vv = (x[table[b].long()].view(L, D).double() for x in (k, v))
        qq = q[b].double()
        s = scale * (qq @ kk.T)
        w = torch.softmax(s, -1)
        delta = (2 * D * 2.0 ** -24 * scale * (qq.abs() @ kk.abs().T) + 2.0 ** -20 * (s.abs() + 64)).amax(-1)
        want.append(w @ vv)
        tol.append((2.0 ** -12 + 4 * delta)[:, None] * (w @ vv.abs()) +
                   2.0 ** -39 * w.amax(-1)[:, None] * vv.abs().sum(0)[None])
    want, tol = torch.stack(want), torch.stack(tol)
    with PagedDecodeAttention(G, 1, D, bs, dt, max_batch=B, max_blocks_per_seq=L // bs) as attn:
        for splits in (1, 0, 3):
            for out_dtype in (torch.float32, dt):
                out = attn.run(q, k, v, table, lens, scale, num_splits=splits, out_dtype=out_dtype).double()
                over = (out - want).abs() - tol - torch.finfo(out_dtype).eps / 2 * want.abs() - 2.0 ** -25
                assert float(over.max()) <= 0, (splits, out_dtype, float((out - want).abs().max()))
        assert attn.check_device_error() == (0, 0)
