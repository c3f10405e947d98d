"""How the append kernel of the block-scaled FP8 cache shares out its work
(csrc/kv_fp8.cu, unit_sequence and the checks behind it), restated for the host:
which block of which sequence every work unit takes, for cu_rows that ascend as
they should and for any others."""
import numpy as np
import pytest

INT_MAX = 2 ** 31 - 1


def unit_sequence(cu, B, bs, u):
    """The 32-way search; None where it finds no sequence."""
    lo, n = 0, B
    while True:
        step = (n + 31) >> 5
        lanes = [i for i in range(0, 32 * step, step) if i < n]
        count = sum(int(cu[lo + i]) // bs + lo + i <= u for i in lanes)
        if count == 0:
            return None
        b = lo + (count - 1) * step
        assert 0 <= b < B
        if step == 1:
            return b
        n = min(step, n - (count - 1) * step)
        lo = b


def pieces(cu, lens, T, bs, max_blocks):
    """[(sequence, page, offset in the block, first row, rows)] over all units, and the sequences
    reported."""
    B = len(lens)
    got, reported = [], set()
    for u in range(T // bs + B):
        if u < B and (cu[u] < 0 or cu[u + 1] < cu[u] or cu[u + 1] > T):
            reported.add(u)
        b = unit_sequence(cu, B, bs, u)
        if b is None:
            continue
        r_lo, r_hi, length = int(cu[b]), int(cu[b + 1]), int(lens[b])
        n = r_hi - r_lo
        base = r_lo // bs + b
        slots = r_hi // bs + b + 1 - base
        j = u - base
        if n <= 0 or j < 0 or j >= slots or r_lo < 0 or r_hi > T:
            continue
        if n > length or length > INT_MAX - bs or length > max_blocks * bs:
            reported.add(b)
            continue
        start, last = length - n, (length - 1) // bs
        page = start // bs + j
        while page <= last:
            t_lo, t_hi = max(start, page * bs), min(length, (page + 1) * bs)
            got.append((b, page, t_lo - page * bs, r_lo + t_lo - start, t_hi - t_lo))
            if j != slots - 1:
                break
            page += 1
    return got, reported


def check_in_bounds(got, cu, lens, T, bs, max_blocks):
    for b, page, off, row, rows in got:
        assert 0 <= b < len(lens)
        assert 0 <= page < max_blocks and 0 <= off < bs
        assert rows >= 1 and off + rows <= bs
        assert 0 <= row and row + rows <= T
        assert cu[b] <= row and row + rows <= cu[b + 1] and row - cu[b] + lens[b] - (cu[b + 1] - cu[b]) == page * bs + off
    assert len({x[:2] for x in got}) == len(got)  # no block twice


@pytest.mark.parametrize("bs", [16, 32, 64])
def test_ascending_rows_cover_every_block_once(bs):
    rng = np.random.default_rng(bs)
    for _ in range(150):
        B = int(rng.choice([1, 2, 5, 31, 32, 33, 70, 1100]))
        new = rng.integers(0, rng.choice([2, 3, 40, 300 if B < 100 else 3]), B)
        cu = np.concatenate([[0], np.cumsum(new)]) + int(rng.integers(0, 3))
        before = rng.integers(0, 100, B)
        lens, T = before + new, int(cu[-1]) + int(rng.integers(0, 3))
        max_blocks = int(lens.max()) // bs + 2
        got, reported = pieces(cu, lens, T, bs, max_blocks)
        check_in_bounds(got, cu, lens, T, bs, max_blocks)
        assert not reported
        want = {(b, page) for b in range(B) if new[b]
                for page in range(int(before[b]) // bs, (int(lens[b]) - 1) // bs + 1)}
        assert {x[:2] for x in got} == want
        assert sum(x[4] for x in got) == int(new.sum())


def descending_arrays():
    yield [320, 480, 0, 16], [160, 16, 16], 480, 16
    yield [0, 40, 8, 60], [50, 40, 60], 60, 16
    yield [0, 10, 8, 25], [20, 30, 40], 25, 16
    rng = np.random.default_rng(1)
    for i in range(1500):
        bs = int(rng.choice([16, 32, 64]))
        B = int(rng.choice([1, 2, 3, 8, 32, 33, 64, 200]))
        T = int(rng.integers(1, 1500))
        kind = i % 4
        if kind == 0:    # anything inside the input
            cu = rng.integers(0, T + 1, B + 1)
        elif kind == 1:  # one descent in an ascending array
            cu = np.sort(rng.integers(0, T + 1, B + 1))
            cu[rng.integers(0, B + 1)] = rng.integers(0, T + 1)
        elif kind == 2:  # outside the input, too
            cu = rng.integers(-2 * T, 3 * T, B + 1)
        else:            # 64-bit garbage
            cu = rng.integers(-2 ** 62, 2 ** 62, B + 1)
        yield cu.tolist(), rng.integers(-5, T + 200, B).tolist(), T, bs


def test_other_rows_stay_in_bounds_and_are_reported():
    for cu, lens, T, bs in descending_arrays():
        max_blocks = max(1, max(lens) // bs)
        got, reported = pieces(cu, lens, T, bs, max_blocks)
        check_in_bounds(got, cu, lens, T, bs, max_blocks)
        bad = {b for b in range(len(lens)) if cu[b] < 0 or cu[b + 1] < cu[b] or cu[b + 1] > T}
        assert bad <= reported
        assert not bad & {x[0] for x in got}
