"""The block-scaled FP8 cache in plain 64-bit numpy: the definition the GPU
tests compare with. Values are float64; caches are E4M3 bytes."""
from __future__ import annotations

import math

import numpy as np

MIN_EXP = -60


def _e4m3_values() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        if c & 0x7F == 0x7F:
            x = math.nan
        v[c] = -x if c & 0x80 else x
    return v


E4M3 = _e4m3_values()


def decode(codes: np.ndarray) -> np.ndarray:
    return E4M3[codes]


def encode(x: np.ndarray) -> np.ndarray:
    """E4M3 bytes of float64 values, to nearest, ties to even, |x| <= 448 (beyond: saturated);
    non-finite: NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    grid = E4M3[:127]                                # 0 .. 448, ascending
    a_ok = np.where(np.isfinite(x), a, 0.0)
    hi = np.searchsorted(grid, a_ok, side="left")    # first grid value >= a
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a_ok - grid[lo], grid[hi] - a_ok
    pick_lo = (d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0))
    code = np.where(pick_lo, lo, hi).astype(np.uint8)
    code = np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def block_scale(x: np.ndarray) -> float:
    """2^e, the smallest e >= -60 with max finite |x| <= 448 * 2^e."""
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    e = MIN_EXP
    if top > 0.0:
        e = max(e, math.frexp(top)[1] - 10)
        while math.ldexp(448.0, e) < top:
            e += 1
    return math.ldexp(1.0, e)


def append(rows: np.ndarray, cache: np.ndarray, scale: np.ndarray, table, lens, cu,
           live: np.ndarray | None = None) -> None:
    """In place. rows [T, Hkv, D] float64, cache [nb, bs, Hkv, D] uint8, scale [nb, Hkv] float32;
    live [T]: rows that are written."""
    nb, bs, Hkv, D = cache.shape
    for b in range(len(lens)):
        r, end = int(cu[b]), int(cu[b + 1])
        pos = int(lens[b]) - (end - r)
        while r < end:
            blk, off = int(table[b][pos // bs]), pos % bs
            n = min(bs - off, end - r)
            ok = np.ones(n, bool) if live is None else live[r:r + n]
            for h in range(Hkv):
                x = rows[r:r + n, h]
                s = block_scale(x[ok])
                if off:
                    old = float(scale[blk, h])
                    if not (old > 0 and math.isfinite(old)):
                        old = 0.0
                    s = max(s, old)
                    if s > old:
                        f = float(np.float32(old) / np.float32(s))
                        y = (decode(cache[blk, :off, h]).astype(np.float32) *
                             np.float32(f)).astype(np.float64)
                        cache[blk, :off, h] = encode(y)
                scale[blk, h] = s
                q = (x.astype(np.float32) / np.float32(s)).astype(np.float64)
                cache[blk, off:off + n, h][ok] = encode(q)[ok]
            r, pos = r + n, pos + n


def gather(cache, scale, table, lens) -> list:
    """Per sequence [len, Hkv, D] float64 values (fp32 products, exact for power-of-two scales)."""
    nb, bs, Hkv, D = cache.shape
    out = []
    for b, L in enumerate(lens):
        blk = np.asarray(table[b])[:-(-int(L) // bs)]
        x = decode(cache[blk]) * scale[blk].astype(np.float64)[:, None, :, None]
        out.append(x.reshape(-1, Hkv, D)[:int(L)])
    return out


def attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale) -> np.ndarray:
    """q [B, Hq, D] float64 -> [B, Hq, D]; an empty context gives zeros."""
    B, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    out = np.zeros(q.shape)
    ks, vs = gather(k_cache, k_scale, table, lens), gather(v_cache, v_scale, table, lens)
    for b in range(B):
        if int(lens[b]) == 0:
            continue
        for hq in range(Hq):
            h = hq // (Hq // Hkv)
            s = ks[b][:, h] @ q[b, hq] * scale
            w = np.exp(s - s.max())
            out[b, hq] = (w @ vs[b][:, h]) / w.sum()
    return out
