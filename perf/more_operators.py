"""Benchmark cases of decode attention over shared prefixes, of capped and biased scores, and of
rotary positions with several axes.

The cache is paged ([num_blocks, block_size, Hkv, D], reached through a block table), 16-bit.

  prefix  decode attention of one query per sequence; runs of consecutive sequences have their first
          tokens in common, in the same blocks of the cache (a system prompt, samples of one prompt)
  scored  decode attention whose scores s = scale * q.k are capped, s' = c tanh(s / c), then get a
          bias slope[head] * (t - (L - 1)) for the distance of token t from the last one, and are
          masked for t < L - window
  rope    rotary positions on q and k, where pair j of a head turns by the position of the token on
          axis[j] (time, height, width), and the paged write of k and v

Cap and distance bias are part of some `prefix` cases too.
"""
import math
import random

import torch

own = False  # False: elementary torch operations; True: the library's kernels

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


def listed():
    return [
        # chat turns behind one long system prompt, 64/8 heads
        dict(name="prefix_system", op="prefix", batch=64, hq=64, hkv=8, d=128, bs=16, dtype="bf16", lens=1, groups=1, plo=8192, phi=8192, lo=1, hi=1024, cap=0.0, alibi=False),
        # a large batch over one document
        dict(name="prefix_document", op="prefix", batch=128, hq=64, hkv=8, d=128, bs=32, dtype="bf16", lens=2, groups=1, plo=16384, phi=16384, lo=64, hi=512, cap=0.0, alibi=False),
        # eight samples of one prompt, a few tokens on: latency
        dict(name="prefix_samples", op="prefix", batch=8, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lens=3, groups=1, plo=1500, phi=1500, lo=1, hi=200, cap=0.0, alibi=False),
        # several prompts of odd lengths, a small model: 14/2 heads of 64
        dict(name="prefix_groups", op="prefix", batch=37, hq=14, hkv=2, d=64, bs=16, dtype="fp16", lens=4, groups=5, plo=0, phi=5003, lo=1, hi=777, cap=0.0, alibi=False),
        # few-shot prompts of a model that caps its scores, 32/4 heads
        dict(name="prefix_capped", op="prefix", batch=24, hq=32, hkv=4, d=128, bs=16, dtype="bf16", lens=5, groups=3, plo=1000, phi=4100, lo=1, hi=300, cap=50.0, alibi=False),
        # long contexts of a small batch with capped scores, 32/8 heads
        dict(name="scored_long", op="scored", batch=4, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lens=6, lo=32768, hi=32768, cap=50.0, alibi=False, window=0),
        # a serving batch of mixed contexts, 64/8 heads, capped
        dict(name="scored_serving", op="scored", batch=96, hq=64, hkv=8, d=128, bs=32, dtype="bf16", lens=7, lo=32, hi=4096, cap=30.0, alibi=False, window=0),
        # a distance bias over a ragged batch from one token on, groups of 7
        dict(name="scored_alibi", op="scored", batch=13, hq=28, hkv=4, d=128, bs=64, dtype="fp16", lens=8, lo=1, hi=9001, cap=0.0, alibi=True, window=0),
        # one user of a small model, a layer with a sliding window: latency
        dict(name="scored_window", op="scored", batch=1, hq=14, hkv=2, d=64, bs=16, dtype="bf16", lens=9, lo=2501, hi=2501, cap=50.0, alibi=False, window=1024),
        # prefill of prompts with images: sections of the rotary pairs for time, height and width
        dict(name="rope_images", op="rope", tokens=16384, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lens=10, rot=128, neox=True, axes=3, mixed=False),
        # video tokens, odd count, half of each head turns, axes interleaved
        dict(name="rope_video", op="rope", tokens=5003, hq=28, hkv=4, d=128, bs=32, dtype="fp16", lens=11, rot=64, neox=False, axes=3, mixed=True),
        # a decode step's new tokens
        dict(name="rope_decode", op="rope", tokens=64, hq=14, hkv=2, d=64, bs=16, dtype="bf16", lens=12, rot=64, neox=True, axes=3, mixed=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "scored", "scored", "rope"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.randint(1, 8 if hkv == 8 else 16)
    case = dict(op=op, hq=hkv * group, hkv=hkv, d=rng.choice([64, 128]), bs=rng.choice([16, 32] if group > 8 else [16, 32, 64]),
                dtype=rng.choice(["bf16", "fp16"]), lens=rng.randrange(1 << 20))
    if op == "rope":
        case.update(tokens=_log_int(rng, 1, 16384), rot=rng.choice([case["d"], case["d"], case["d"] // 2]), neox=rng.random() < 0.5,
                    axes=rng.choice([2, 3, 3]), mixed=rng.random() < 0.5)
        case["hq"] = hkv * min(group, 8)
        return case
    batch = _log_int(rng, 1, 128)
    case.update(batch=batch, cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.25)
    if op == "prefix":
        phi = _log_int(rng, 16, 16384)
        case.update(groups=rng.randint(1, min(batch, 6)), plo=rng.choice([0, phi, max(1, phi // 2)]), phi=phi,
                    lo=rng.choice([0, 1]), hi=_log_int(rng, 2, 32768 // max(16, batch)))
    else:
        if not case["alibi"] and case["cap"] == 0.0:
            case["cap"] = 20.0
        hi = _log_int(rng, 16, 65536 // max(2, batch))
        case.update(lo=rng.choice([0, 1, max(1, hi // 2)]), hi=hi, window=rng.choice([0, 0, _log_int(rng, 1, 4096)]))
    return case


def _sizes(case):
    """(prefix tokens of each run of sequences, first sequence of each run, whole context of each sequence)."""
    rng = random.Random(case["lens"])
    batch, lo, hi = case["batch"], case["lo"], case["hi"]
    mine = [_log_int(rng, max(1, lo), hi) if hi > 1 else hi for _ in range(batch)]
    if lo == 0:
        mine[rng.randrange(batch)] = 0
    if case["op"] == "scored":
        return [], [0], mine
    plo, phi, groups = case["plo"], case["phi"], case["groups"]
    prefix = [_log_int(rng, max(1, plo), phi) for _ in range(groups)]
    if plo == 0 and groups > 1:
        prefix[rng.randrange(groups)] = 0
    cuts = [0] + sorted(rng.sample(range(1, batch), groups - 1)) + [batch]
    whole = []
    for i, p in enumerate(prefix):
        whole += [p + x for x in mine[cuts[i]:cuts[i + 1]]]
    return prefix, cuts, whole


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _slopes(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1, dtype=torch.float64, device=DEV) / hq).float()


def _axes(case):
    """The axis of each rotary pair: sections of about equal size, one after the other or in turns."""
    pairs, n = case["rot"] // 2, case["axes"]
    if case["mixed"]:
        return [j % n for j in range(pairs)]
    return [min(n - 1, j * n // pairs) for j in range(pairs)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + case["lens"])
    hq, hkv, d, bs, dtype = case["hq"], case["hkv"], case["d"], case["bs"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "rope":
        t = case["tokens"]
        blocks = -(-t // bs) + 4
        qkv = _normal(gen, t, hq + 2 * hkv, d).to(dtype)  # one projection's output; q, k, v are views
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        side = max(1, math.isqrt(max(1, t // 4)))
        at = torch.arange(t, device=DEV)
        grid = torch.stack([at // (side * side), at // side % side, at % side])[:case["axes"]]
        s["positions"] = (grid + torch.randint(0, 1000, (1,), generator=gen, device=DEV)).to(torch.int32)
        half = case["rot"] // 2
        inv = torch.pow(1000000.0, -torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = torch.arange(1000 + t, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["slots"] = torch.randperm(blocks * bs, generator=gen, device=DEV)[:t]
        s["k_cache"], s["v_cache"] = (_normal(gen, blocks, bs, hkv, d).to(dtype) for _ in range(2))
        s["q_out"] = torch.empty(t, hq, d, dtype=dtype, device=DEV)
        s["axis"] = _axes(case)
        return s
    prefix, cuts, whole = _sizes(case)
    batch = case["batch"]
    shared = [p // bs for p in prefix]
    first = [0] * batch  # a sequence's blocks that it shares
    for i, n in enumerate(shared):
        first[cuts[i]:cuts[i + 1]] = [n] * (cuts[i + 1] - cuts[i])
    pages = [-(-x // bs) for x in whole]
    used = sum(shared) + sum(max(0, n - f) for n, f in zip(pages, first))
    num_blocks, width = used + used // 8 + 4, max(1, max(pages))
    order = torch.randperm(num_blocks, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(batch, width, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(shared):
        table[cuts[i]:cuts[i + 1], :n] = order[at:at + n]
        at += n
    for b, n in enumerate(pages):
        table[b, first[b]:n] = order[at:at + n - first[b]]
        at += n - first[b]
    s["table"], s["lens"] = table, torch.tensor(whole, dtype=torch.int32, device=DEV)
    for name in ("k_cache", "v_cache"):
        s[name] = torch.empty(num_blocks, bs, hkv, d, dtype=dtype, device=DEV)
        s[name].copy_(_normal(gen, num_blocks, bs, hkv, d))
    s["q"] = (1.5 * _normal(gen, batch, hq, d)).to(dtype)
    s["scale"] = 1.0 / math.sqrt(d)
    s["slopes"] = _slopes(hq) if case["alibi"] else None
    if prefix:
        s["cu_seqs"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device=DEV)
    if own:
        from paged_gqa_decode_attention_gb300 import PagedDecodeAttention
        s["handle"] = PagedDecodeAttention(hq, hkv, d, bs, dtype, max_batch=batch, max_blocks_per_seq=width)
    return s


def work(case):
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    if case["op"] == "rope":
        t = case["tokens"]
        rows = min(t * case["axes"], 1000 + t)
        return {"bytes": 4 * t * (hq + 2 * hkv) * d + 4 * t * case["axes"] + 8 * t + 4 * rows * case["rot"],
                "flops": 3 * t * (hq + hkv) * case["rot"]}
    prefix, cuts, whole = _sizes(case)
    window = case.get("window", 0)
    seen = [min(x, window) if window else x for x in whole]
    read = sum(seen)
    for i, p in enumerate(prefix):  # a shared block is read once
        read -= (cuts[i + 1] - cuts[i] - 1) * (p // bs * bs)
    return {"bytes": 4 * read * hkv * d + 4 * (read // bs + len(whole)) + 4 * len(whole) * hq * d + 4 * len(whole),
            "flops": 4 * sum(seen) * hq * d}


# ------------------------------ plain forms ------------------------------

def _attn_plain(s):
    case, table, lens = s["case"], s["table"].long(), s["lens"].long()
    batch, hkv, d = case["batch"], case["hkv"], case["d"]
    q = s["q"].float().view(batch, hkv, -1, d)
    k = s["k_cache"][table].float().view(batch, -1, hkv, d).transpose(1, 2)
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    if case["cap"]:
        score = case["cap"] * torch.tanh(score / case["cap"])
    t = torch.arange(score.shape[-1], device=DEV)[None, :]
    if s["slopes"] is not None:
        far = (t - (lens[:, None] - 1)).float()
        score = score + s["slopes"].view(1, hkv, -1, 1) * far[:, None, None, :]
    held = t < lens[:, None]
    if case.get("window", 0):
        held = held & (t >= lens[:, None] - case["window"])
    score = score.masked_fill(~held[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][table].float().view(batch, -1, hkv, d).transpose(1, 2)
    out = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return out.view(batch, -1, d).to(s["q"].dtype)


def _rotated(s, x):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    axis = torch.tensor(s["axis"], device=DEV)
    pair = torch.arange(half, device=DEV)
    where = s["positions"].long()[axis].T  # [tokens, pairs]
    c, t = s["cos_sin"][where, pair].double()[:, None, :], s["cos_sin"][where, half + pair].double()[:, None, :]
    x64 = x.double()
    a, b = (x64[..., :half], x64[..., half:rot]) if case["neox"] else (x64[..., 0:rot:2], x64[..., 1:rot:2])
    ya, yb = a * c - b * t, b * c + a * t
    y = torch.cat([ya, yb], -1) if case["neox"] else torch.stack([ya, yb], -1).flatten(-2)
    return torch.cat([y, x64[..., rot:]], -1).to(x.dtype)


def run(s):
    case = s["case"]
    if own:
        if case["op"] == "rope":
            import paged_gqa_decode_attention_gb300 as pda
            q_out = pda.rope_axes_kv_write(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["k_cache"],
                                           s["v_cache"], s["axis"], neox=case["neox"], q_out=s["q_out"])
            return q_out, s["k_cache"], s["v_cache"]
        more = dict(scale=s["scale"], softcap=case["cap"], alibi_slopes=s["slopes"])
        if case["op"] == "prefix":
            return s["handle"].run_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu_seqs"],
                                                 s["prefix_lens"], **more)
        return s["handle"].run(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], window=case["window"], **more)
    if case["op"] != "rope":
        return _attn_plain(s)
    q_out = _rotated(s, s["q"])
    shape = s["k_cache"].shape
    s["k_cache"].view(-1, *shape[2:])[s["slots"]] = _rotated(s, s["k"])
    s["v_cache"].view(-1, *shape[2:])[s["slots"]] = s["v"]
    return q_out, s["k_cache"], s["v_cache"]


# ------------------------- the definition, in 64 bits -------------------------

def exact(case, seed):
    s = prepare(case, seed)
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    if case["op"] == "rope":
        half = case["rot"] // 2
        cs = s["cos_sin"].double()

        def turned(x):
            y = x.double().clone()
            for j, axis in enumerate(s["axis"]):
                i, k = (j, j + half) if case["neox"] else (2 * j, 2 * j + 1)
                row = cs[s["positions"][axis].long()]
                c, t = row[:, j, None], row[:, half + j, None]
                a, b = x[..., i].double(), x[..., k].double()
                y[..., i], y[..., k] = a * c - b * t, a * t + b * c
            return y

        out = []
        for cache, rows in ((s["k_cache"], turned(s["k"])), (s["v_cache"], s["v"].double())):
            flat = cache.double().view(-1, hkv, d)
            flat[s["slots"]] = rows
            out.append(flat.view(cache.shape))
        return turned(s["q"]), out[0], out[1]
    window = case.get("window", 0)
    group = case["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        start = max(0, n - window) if window else 0
        if n == start:
            continue
        blk = s["table"][b, start // bs:-(-n // bs)].long()
        rows = slice(start % bs, start % bs + n - start)
        k = s["k_cache"][blk].reshape(-1, hkv, d)[rows].double()
        v = s["v_cache"][blk].reshape(-1, hkv, d)[rows].double()
        q = s["q"][b].double().view(hkv, group, d)
        score = torch.einsum("hgd,thd->hgt", q, k) * s["scale"]
        if case["cap"]:
            score = case["cap"] * torch.tanh(score / case["cap"])
        if s["slopes"] is not None:
            far = torch.arange(start, n, device=DEV, dtype=torch.float64) - (n - 1)
            score = score + s["slopes"].double().view(hkv, group, 1) * far
        out[b] = torch.einsum("hgt,thd->hgd", torch.softmax(score, -1), v).reshape(-1, d)
    return out
