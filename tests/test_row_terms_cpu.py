"""That the bound of row_terms_ref.py tells weights of one 16-bit term from weights of two."""
import pytest
import torch

from row_terms_ref import OWN, SHARED, make_terms, reference

CASES = ([([n + p for n in own], hq, hkv, d, bs, dt, 0.0, 0) for own, p, hq, hkv, d, bs, dt in SHARED] + OWN)


@pytest.mark.parametrize("lens,hq,hkv,d,bs,dtype,cap,window", CASES)
def test_one_term_is_out_of_bounds(lens, hq, hkv, d, bs, dtype, cap, window):
    lens = lens[:3]
    args = make_terms(lens, hq, hkv, d, bs, dtype, seed=3)
    want, tol = reference(*args, 1.0, cap, None, window)

    def one(p):  # the rounded weights are divided by the sum of the rounded or of the exact ones
        r = p.to(dtype).double()
        return r, r.sum(-1, keepdim=True)

    def one_of_exact(p):
        return p.to(dtype).double(), p.sum(-1, keepdim=True)

    def two(p):
        r = p.to(dtype).double()
        return r + (p - r).to(dtype).double(), p.sum(-1, keepdim=True)

    for model, fits in ((one, False), (one_of_exact, False), (two, True)):
        got = reference(*args, 1.0, cap, None, window, weights=model)[0].to(dtype).double()
        over = (got - want).abs() > tol
        # each head of each sequence shows it
        assert not over.any() if fits else over.any(-1).all()
