"""Benchmark cases of the block-scaled FP8 KV cache: writing it, reading it back, attending to it.

The cache is paged like the 16-bit one ([num_blocks, block_size, Hkv, D], reached through a block
table) and holds E4M3 values; every block of block_size tokens has one fp32 scale per kv head, for K
and for V ([num_blocks, Hkv] each), and a stored value stands for scale * e4m3.

  append       new rows of k and v are quantised and appended to each sequence's pages
  rope_append  the same after rotary positions on q and k (q_out holds the rotated queries)
  gather       each sequence's tokens are read back as contiguous 16-bit or fp32 rows
  attn         decode attention of one query per sequence over that cache

The scale of a block and head is the power of two 2^e, e >= -60, with the smallest e for which
the largest |x| of the block is at most 448 * 2^e (448: the largest E4M3 value). It never shrinks
while a block fills: a call that appends behind tokens that a block already holds keeps the larger
of the old scale and the one that its own rows need, and where that is larger than the old one the
block's earlier values are rounded again to the new scale. A call that writes a block's first token
starts the block anew. Quantisation rounds to nearest, ties to even.
"""
import math
import random

import torch

own = False  # False: elementary torch operations; True: the library's kernels

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = torch.float8_e4m3fn
MIN_EXP = -60
DEV = "cuda"


def listed():
    return [
        # one long-context decode step of a small batch: 32/8 heads, contexts of 32768 tokens
        dict(name="attn_long", op="attn", batch=4, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lens=1, lo=32768, hi=32768),
        # a serving batch of mixed contexts at 64/8 heads
        dict(name="attn_serving", op="attn", batch=128, hq=64, hkv=8, d=128, bs=32, dtype="bf16", lens=2, lo=32, hi=4096),
        # a ragged batch of odd lengths from one token on, groups of 7, big pages, fp16
        dict(name="attn_ragged", op="attn", batch=13, hq=28, hkv=4, d=128, bs=64, dtype="fp16", lens=3, lo=1, hi=9001),
        # one interactive user of a small model: 14/2 heads of 64, a few hundred tokens; latency
        dict(name="attn_single", op="attn", batch=1, hq=14, hkv=2, d=64, bs=16, dtype="bf16", lens=4, lo=777, hi=777),
        # a decode step's new tokens, one a sequence, anywhere inside their pages
        dict(name="append_decode", op="append", batch=256, hkv=8, d=128, bs=16, dtype="bf16", lens=5, lo=1, hi=1000, new_lo=1, new_hi=1),
        # chunked prefill: ragged chunks behind earlier tokens
        dict(name="append_prefill", op="append", batch=7, hkv=8, d=128, bs=32, dtype="fp16", lens=6, lo=1, hi=3000, new_lo=1111, new_hi=9999),
        # a decode step of a small model with rotary positions, scaled for long contexts
        dict(name="rope_append_decode", op="rope_append", batch=32, hq=14, hkv=2, d=64, bs=16, dtype="bf16", lens=7, lo=1, hi=900, new_lo=1, new_hi=1, rot=64, neox=True, factor=4.0),
        # prefill of four prompts at 32/8 heads
        dict(name="rope_append_prefill", op="rope_append", batch=4, hq=32, hkv=8, d=128, bs=16, dtype="bf16", lens=8, lo=1, hi=64, new_lo=4097, new_hi=8190, rot=128, neox=True, factor=1.0),
        # prefixes read back for a 16-bit attention over them
        dict(name="gather_prefix", op="gather", batch=8, hkv=8, d=128, bs=16, dtype="bf16", lens=9, lo=1000, hi=8191),
        # a few short sequences moved out of the cache, exactly
        dict(name="gather_short", op="gather", batch=3, hkv=2, d=64, bs=32, dtype="fp32", lens=10, lo=5, hi=300),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "rope_append", "gather"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    case = dict(op=op, hkv=hkv, d=d, dtype=rng.choice(["bf16", "fp16"]), lens=rng.randrange(1 << 20))
    if op == "attn":
        group = rng.randint(1, 16)
        batch = _log_int(rng, 1, 128)
        hi = _log_int(rng, 16, 65536 // max(2, batch))
        case.update(batch=batch, hq=group * hkv, bs=rng.choice([16, 32] if group > 8 else [16, 32, 64]),
                    lo=rng.choice([0, 1, max(1, hi // 2)]), hi=hi)
    elif op == "gather":
        batch = _log_int(rng, 1, 64)
        case.update(batch=batch, bs=rng.choice([16, 32, 64]), lo=0, hi=_log_int(rng, 2, 32768 // batch),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    else:
        batch = _log_int(rng, 1, 256)
        new = rng.choice([1, _log_int(rng, 1, max(2, 24000 // batch))])
        case.update(batch=batch, bs=rng.choice([16, 32, 64]), lo=0, hi=_log_int(rng, 2, 1000),
                    new_lo=min(1, new - 1), new_hi=new)
        if op == "rope_append":
            case.update(hq=hkv * rng.randint(1, 8), rot=rng.choice([d, d, d // 2]), neox=rng.random() < 0.5,
                        factor=rng.choice([1.0, 4.0, 8.0]))
    return case


def _sizes(case):
    """(tokens each sequence holds before the call, new tokens of each), from the case alone."""
    rng = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    before = [_log_int(rng, max(1, lo), hi) if hi > 1 else hi for _ in range(case["batch"])]
    if lo == 0:
        before[rng.randrange(len(before))] = 0
    new = [0] * len(before)
    if "new_hi" in case:
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in before]
        if not any(new):
            new[0] = 1
    return before, new


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _rows(gen, t, heads, d):
    """Rows as projections give them: a spread of sizes between tokens, a few channels that stand out."""
    channel = torch.exp2(_normal(gen, heads, d).clamp(-3, 3))
    return _normal(gen, t, heads, d) * channel * torch.exp2(0.7 * _normal(gen, t, heads, 1))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + case["lens"])
    before, new = _sizes(case)
    batch, hkv, d, bs, dtype = case["batch"], case["hkv"], case["d"], case["bs"], DTYPES[case["dtype"]]
    after = [x + y for x, y in zip(before, new)]
    pages = [-(-x // bs) for x in after]
    num_blocks = sum(pages) + sum(pages) // 8 + 4
    width = max(1, max(pages))
    order = torch.randperm(num_blocks, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(batch, width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(case=case, table=table, lens=torch.tensor(after, dtype=torch.int32, device=DEV))
    for name in ("k", "v"):
        x = _rows(gen, num_blocks * bs, hkv, d).view(num_blocks, bs, hkv, d)
        scale = _power(x.abs().amax((1, 3)))
        s[name + "_scale"] = scale
        s[name + "_cache"] = (x / scale[:, None, :, None]).to(FP8)
        del x
    if case["op"] == "attn":
        s["q"] = _normal(gen, batch, case["hq"], d).to(dtype)
        s["scale"] = 1.0 / math.sqrt(d) / 2
        if own:
            from paged_gqa_decode_attention_gb300 import PagedDecodeAttention
            s["handle"] = PagedDecodeAttention(case["hq"], hkv, d, bs, dtype, max_batch=batch,
                                               max_blocks_per_seq=width, kv_fp8=True)
    elif case["op"] == "gather":
        cu = [0]
        for x in before:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int64, device=DEV)
        s["rows"], s["max_len"] = cu[-1], max(before)
        s["k_out"] = torch.empty(cu[-1], hkv, d, dtype=dtype, device=DEV)
        s["v_out"] = torch.empty(cu[-1], hkv, d, dtype=dtype, device=DEV)
    else:
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int64, device=DEV)
        hq = case.get("hq", 0)
        qkv = _rows(gen, cu[-1], hq + 2 * hkv, d).to(dtype)  # one projection's output; q, k, v are views
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if case["op"] == "rope_append":
            spots = [torch.arange(x, y, device=DEV) for x, y in zip(before, after)]
            s["positions"] = torch.cat(spots).to(torch.int32)
            half = case["rot"] // 2
            inv = torch.pow(10000.0, -torch.arange(half, dtype=torch.float64, device=DEV) / half)
            angle = torch.arange(max(after) + 1, dtype=torch.float64, device=DEV)[:, None] / case["factor"] * inv
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
            s["q_out"] = torch.empty(cu[-1], hq, d, dtype=dtype, device=DEV)
    return s


def work(case):
    before, new = _sizes(case)
    hkv, d, bs, batch = case["hkv"], case["d"], case["bs"], case["batch"]
    esz = 4 if case["dtype"] == "fp32" else 2
    tokens = sum(before)
    if case["op"] == "attn":
        pages = sum(-(-x // bs) for x in before)
        return {"bytes": 2 * tokens * hkv * d + 8 * pages * hkv + 4 * pages + 4 * batch + 4 * batch * case["hq"] * d,
                "flops": 4 * tokens * case["hq"] * d}
    if case["op"] == "gather":
        pages = sum(-(-x // bs) for x in before)
        return {"bytes": 2 * tokens * hkv * d * (1 + esz) + 8 * pages * hkv + 4 * pages + 12 * batch,
                "flops": 2 * tokens * hkv * d}
    rows = sum(new)
    pages = sum(-(-(x + y) // bs) - x // bs for x, y in zip(before, new) if y)
    bytes_ = 2 * rows * hkv * d * 3 + 8 * pages * hkv + 4 * pages + 12 * batch
    flops = 6 * rows * hkv * d
    if case["op"] == "rope_append":
        hq = case["hq"]
        bytes_ += 2 * rows * hq * d * 2 + 4 * rows + 4 * min(rows, max(before) + max(new)) * case["rot"]
        flops += 3 * rows * (hq + hkv) * case["rot"]
    return {"bytes": bytes_, "flops": flops}


# ------------------------------ plain forms ------------------------------

def _power(amax):
    """The scale of a block whose largest magnitude is amax (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    x = torch.where(m <= 0.875, e - 9, e - 8)
    x = torch.where(amax > 0, x, MIN_EXP).clamp(min=MIN_EXP)
    return torch.exp2(x.double()).float()


def _round16(x, dtype):
    """float64 rounded once to a 16-bit type (a cast rounds to 32 bits first)."""
    bits, low = (8, -125) if dtype == torch.bfloat16 else (11, -13)
    _, e = torch.frexp(x)
    step = torch.exp2((e.clamp(min=low) - bits).double())
    return (torch.round(x / step) * step).to(dtype)


def _rotated(x, cos_sin, positions, rot, neox):
    x64 = x.double()
    half = rot // 2
    cs = cos_sin[positions.long()].double()[:, None, :]
    c, s = cs[..., :half], cs[..., half:]
    a, b = (x64[..., :half], x64[..., half:rot]) if neox else (x64[..., 0:rot:2], x64[..., 1:rot:2])
    ya, yb = a * c - b * s, b * c + a * s
    y = torch.cat([ya, yb], -1) if neox else torch.stack([ya, yb], -1).flatten(-2)
    return _round16(torch.cat([y, x64[..., rot:]], -1), x.dtype)


def _places(s, first, total, lens_before):
    """Sequence, block and slot in the block of every row."""
    row = torch.arange(total, device=DEV)
    b = torch.searchsorted(first, row, right=True) - 1
    pos = lens_before[b] + row - first[b]
    bs = s["case"]["bs"]
    return s["table"].long()[b, pos // bs], pos % bs


def _quantise_into(x, cache, scale, blk, off, blk0, keep):
    x = x.float()
    amax = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    touched = torch.zeros(scale.shape[0], 1, dtype=torch.bool, device=DEV)
    touched[blk] = True
    fresh = torch.ones_like(touched)
    fresh[blk0] = (keep == 0)[:, None]
    old = torch.where(fresh, torch.zeros_like(scale), scale)
    new = torch.where(touched, torch.maximum(old, _power(amax)), scale)
    raw = cache.view(torch.uint8)
    page = raw[blk0]
    again = (page.view(FP8).float() * (scale / new)[blk0][:, None, :, None]).to(FP8).view(torch.uint8)
    held = torch.arange(cache.shape[1], device=DEV)[None, :] < keep[:, None]
    raw[blk0] = torch.where(held[:, :, None, None], again, page)
    raw[blk, off] = (x / new[blk][:, :, None]).to(FP8).view(torch.uint8)
    scale.copy_(new)


def _append_plain(s, k, v):
    cu, bs = s["cu"], s["case"]["bs"]
    n = cu[1:] - cu[:-1]
    start = s["lens"].long() - n
    blk, off = _places(s, cu, k.shape[0], start)
    width = s["table"].shape[1]
    blk0 = s["table"].long()[torch.arange(n.shape[0], device=DEV), (start // bs).clamp(max=width - 1)]
    _quantise_into(k, s["k_cache"], s["k_scale"], blk, off, blk0, start % bs)
    _quantise_into(v, s["v_cache"], s["v_scale"], blk, off, blk0, start % bs)


def _attn_plain(s):
    case, table, lens = s["case"], s["table"].long(), s["lens"].long()
    batch, hkv, d = case["batch"], case["hkv"], case["d"]
    def values(name):
        x = s[name + "_cache"].view(torch.uint8)[table].view(FP8).float() * s[name + "_scale"][table][:, :, None, :, None]
        return x.view(batch, -1, hkv, d).transpose(1, 2)
    q = s["q"].float().view(batch, hkv, -1, d)
    k = values("k")
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    held = (torch.arange(score.shape[-1], device=DEV)[None, :] < lens[:, None])[:, None, None, :]
    score = score.masked_fill(~held, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values("v")) / torch.where(total == 0, torch.ones_like(total), total)
    return out.view(batch, -1, d).to(s["q"].dtype)


def _gather_plain(s):
    blk, off = _places(s, s["cu"], s["rows"], torch.zeros_like(s["lens"]).long())
    def values(name):
        x = s[name + "_cache"].view(torch.uint8)[blk, off].view(FP8).float() * s[name + "_scale"][blk][:, :, None]
        return x.to(s["k_out"].dtype)
    return values("k"), values("v")


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import paged_gqa_decode_attention_gb300 as pda
        if op == "attn":
            return s["handle"].run(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["scale"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op == "gather":
            return pda.gather_kv_fp8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                                     cu_rows=s["cu"][:-1], max_len=s["max_len"], k_out=s["k_out"], v_out=s["v_out"])
        if op == "append":
            pda.append_kv_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                              s["lens"], s["cu"])
            return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        q_out = pda.rope_append_kv_fp8(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"],
                                       s["k_scale"], s["v_scale"], s["table"], s["lens"], s["cu"], neox=case["neox"],
                                       q_out=s["q_out"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], q_out
    if op == "attn":
        return _attn_plain(s)
    if op == "gather":
        return _gather_plain(s)
    if op == "append":
        _append_plain(s, s["k"], s["v"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    q_out = _rotated(s["q"], s["cos_sin"], s["positions"], case["rot"], case["neox"])
    _append_plain(s, _rotated(s["k"], s["cos_sin"], s["positions"], case["rot"], case["neox"]), s["v"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], q_out


# ------------------------- the definition, in 64 bits -------------------------

def _e4m3(codes):
    """The value of every E4M3 byte: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    value = torch.tensor([(-1.0) ** (c >> 7) * (math.ldexp(c & 7, -9) if (c >> 3) & 15 == 0 else
                                               math.ldexp(8 + (c & 7), ((c >> 3) & 15) - 10)) for c in range(256)],
                         dtype=torch.float64, device=DEV)
    return value[codes.view(torch.uint8).int()]


def _to_grid(y, digits, lowest):
    """y rounded to `digits` significant bits, ties to even, its last bit at least 2^lowest."""
    last = torch.floor(torch.log2(y.abs().clamp(min=1e-300))) - (digits - 1)
    unit = torch.exp2(last.clamp(min=lowest))
    return torch.round(y / unit) * unit


def _exact_scale(x):
    """[Hkv] scales for values x [tokens, Hkv, D]."""
    got = []
    for top in x.abs().amax((0, 2)).tolist():
        e = MIN_EXP
        if top > 0:
            e = max(e, math.ceil(math.log2(top / 448.0)) - 1)
            while top > 448.0 * 2.0 ** e:
                e += 1
        got.append(2.0 ** e)
    return torch.tensor(got, dtype=torch.float64, device=DEV)


def _exact_append(s, rows, name):
    bs, table = s["case"]["bs"], s["table"].tolist()
    value, scale = _e4m3(s[name + "_cache"]), s[name + "_scale"].double()
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b, total in enumerate(lens):
        at, end = cu[b], cu[b + 1]
        pos = total - (end - at)
        while at < end:
            blk, off = table[b][pos // bs], pos % bs
            n = min(bs - off, end - at)
            new = rows[at:at + n].double()
            need = _exact_scale(new)
            if off:
                need = torch.maximum(need, scale[blk])
                value[blk, :off] = _to_grid(value[blk, :off] * (scale[blk] / need)[None, :, None], 4, -9)
            scale[blk] = need
            value[blk, off:off + n] = _to_grid(new / need[None, :, None], 4, -9)
            at, pos = at + n, pos + n
    return value, scale


def _exact_rope(s, x):
    case = s["case"]
    rot, digits, lowest = case["rot"], *((8, -133) if x.dtype == torch.bfloat16 else (11, -24))
    y = x.double().clone()
    table = s["cos_sin"].double()[s["positions"].long()]
    for j in range(rot // 2):
        i, k = (j, j + rot // 2) if case["neox"] else (2 * j, 2 * j + 1)
        c, t = table[:, j, None], table[:, rot // 2 + j, None]
        a, b = x[..., i].double(), x[..., k].double()
        y[..., i], y[..., k] = _to_grid(a * c - b * t, digits, lowest), _to_grid(a * t + b * c, digits, lowest)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("append", "rope_append"):
        k = _exact_rope(s, s["k"]) if op == "rope_append" else s["k"]
        kc, ks = _exact_append(s, k, "k")
        vc, vs = _exact_append(s, s["v"], "v")
        return (kc, vc, ks, vs) + ((_exact_rope(s, s["q"]),) if op == "rope_append" else ())
    bs, hkv, d = case["bs"], case["hkv"], case["d"]
    lens = s["lens"].tolist()

    def tokens(name, b):
        blk = s["table"][b, :-(-lens[b] // bs)].long()
        x = _e4m3(s[name + "_cache"].view(torch.uint8)[blk]) * s[name + "_scale"][blk].double()[:, None, :, None]
        return x.reshape(-1, hkv, d)[:lens[b]]

    if op == "gather":
        return tuple(torch.cat([tokens(n, b) for b in range(len(lens))]) for n in ("k", "v"))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    group = case["hq"] // hkv
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = tokens("k", b), tokens("v", b)
        for h in range(hkv):
            heads = slice(h * group, (h + 1) * group)
            weight = torch.softmax(s["q"][b, heads].double() @ k[:, h].T * s["scale"], -1)
            out[b, heads] = weight @ v[:, h]
    return out
