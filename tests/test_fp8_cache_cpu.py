"""The block-scaled FP8 cache without a GPU: the 64-bit reference against
independent facts, and the refusals of the entry points before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp8_cache_ref as ref
import paged_gqa_decode_attention_gb300 as pda
from paged_gqa_decode_attention_gb300 import build as pda_build


@pytest.fixture(scope="module")
def lib():
    pda_build.build()
    return pda.load_library()


# ------------------------------ the reference ------------------------------

def test_e4m3_decode_and_encode_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.decode(codes), want)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), np.exp2(rng.uniform(-12, 8.8, 20000)),
                        (ref.E4M3[:126] + ref.E4M3[1:127]) / 2])  # every midpoint
    x = x.astype(np.float32)
    got = ref.encode(x.astype(np.float64))
    np.testing.assert_array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn)
                                  .view(torch.uint8).numpy())


@pytest.mark.parametrize("top,scale", [(448.0, 1.0), (448.5, 2.0), (1.75, 2.0 ** -8),
                                       (1.0, 2.0 ** -8), (0.0, 2.0 ** -60), (1e-30, 2.0 ** -60),
                                       (3.3e38, 2.0 ** 120)])
def test_block_scale_closed_forms(top, scale):
    assert ref.block_scale(np.array([top, -top / 3, math.nan, math.inf])) == scale


def test_stepwise_append_equals_one_call_for_normal_values():
    """A block filled token by token holds what one call writes, unless a raised scale pushed a
    value below E4M3's normal range (2^-6 of the scale)."""
    rng = np.random.default_rng(1)
    x = np.float32(rng.standard_normal((32, 2, 64))).astype(np.float64)
    x += np.copysign(0.25, x)  # |x| in [0.25, 8): exponents well inside E4M3's
    table, a, b = [[1, 0]], np.zeros((2, 16, 2, 64), np.uint8), np.zeros((2, 16, 2, 64), np.uint8)
    sa, sb = np.full((2, 2), np.nan, np.float32), np.full((2, 2), np.nan, np.float32)
    ref.append(x, a, sa, table, [32], [0, 32])
    for t in range(32):
        ref.append(x[t:t + 1], b, sb, table, [t + 1], [0, 1])
    np.testing.assert_array_equal(sa, sb)
    np.testing.assert_array_equal(a, b)


# -------------------------------- refusals ---------------------------------

A = 1 << 20  # an aligned stand-in address; no call below reaches a launch


def append_args(**kw):
    d = dict(k=A, ks=0, v=2 * A, vs=0, T=4, Hkv=2, D=128, dtype=0, kc=3 * A, vc=4 * A, ksc=5 * A,
             vsc=6 * A, nb=4, bs=16, table=7 * A, mb=2, lens=8 * A, cu=9 * A, B=2, err=None, dev=0,
             stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), pda.PDA_EINVAL), (dict(B=-1), pda.PDA_EINVAL), (dict(dev=-1), pda.PDA_EINVAL),
    (dict(T=1 << 31), pda.PDA_EINVAL), (dict(dtype=2), pda.PDA_EINVAL),
    (dict(Hkv=0), pda.PDA_EINVAL), (dict(D=0), pda.PDA_EINVAL), (dict(D=96), pda.PDA_EUNSUPPORTED),
    (dict(D=256), pda.PDA_EUNSUPPORTED), (dict(bs=8), pda.PDA_EUNSUPPORTED),
    (dict(bs=128), pda.PDA_EUNSUPPORTED), (dict(nb=0), pda.PDA_EINVAL),
    (dict(nb=1 << 28), pda.PDA_EINVAL), (dict(ks=128), pda.PDA_EINVAL),
    (dict(vs=260), pda.PDA_EINVAL), (dict(k=None), pda.PDA_EINVAL), (dict(cu=None), pda.PDA_EINVAL),
    (dict(ksc=None), pda.PDA_EINVAL), (dict(mb=0), pda.PDA_EINVAL), (dict(k=A + 8), pda.PDA_EINVAL),
    (dict(kc=3 * A + 1), pda.PDA_EINVAL), (dict(cu=9 * A + 4), pda.PDA_EINVAL),
    (dict(vsc=6 * A + 2), pda.PDA_EINVAL), (dict(vc=3 * A), pda.PDA_EALIAS),
    (dict(kc=A), pda.PDA_EALIAS), (dict(ksc=8 * A), pda.PDA_EALIAS),
    (dict(vsc=5 * A), pda.PDA_EALIAS), (dict(err=5 * A), pda.PDA_EALIAS),
    (dict(T=0), pda.PDA_OK), (dict(B=0, cu=None), pda.PDA_OK),
])
def test_append_refusals_before_cuda(lib, kw, status):
    assert lib.paged_decode_attn_append_kv_fp8(*append_args(**kw)) == status
    if status != pda.PDA_OK:
        assert lib.paged_decode_attn_last_error()


def rope_args(**kw):
    d = dict(q=10 * A, qs=0, k=A, ks=0, v=2 * A, vs=0, pos=11 * A, cs=12 * A, maxpos=64, rot=64,
             neox=1, T=4, Hq=4, Hkv=2, D=128, dtype=0, qo=13 * A, qos=0, kc=3 * A, vc=4 * A,
             ksc=5 * A, vsc=6 * A, nb=4, bs=16, table=7 * A, mb=2, lens=8 * A, cu=9 * A, B=2,
             err=None, dev=0, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=0), pda.PDA_EINVAL), (dict(rot=24), pda.PDA_EINVAL), (dict(rot=144), pda.PDA_EINVAL),
    (dict(rot=-16), pda.PDA_EINVAL), (dict(maxpos=-1), pda.PDA_EINVAL), (dict(q=None), pda.PDA_EINVAL),
    (dict(qo=None), pda.PDA_EINVAL), (dict(pos=None), pda.PDA_EINVAL), (dict(cs=None), pda.PDA_EINVAL),
    (dict(qs=256), pda.PDA_EINVAL), (dict(qos=516), pda.PDA_EINVAL), (dict(pos=11 * A + 2), pda.PDA_EINVAL),
    (dict(qo=10 * A, qos=1024), pda.PDA_EALIAS), (dict(qo=10 * A + 16), pda.PDA_EALIAS),
    (dict(qo=A), pda.PDA_EALIAS), (dict(qo=3 * A), pda.PDA_EALIAS), (dict(kc=10 * A), pda.PDA_EALIAS),
    (dict(dtype=2), pda.PDA_EINVAL), (dict(T=0), pda.PDA_OK),
])
def test_rope_append_refusals_before_cuda(lib, kw, status):
    assert lib.paged_decode_attn_rope_append_kv_fp8(*rope_args(**kw)) == status


def gather_args(**kw):
    d = dict(kc=A, vc=2 * A, ksc=3 * A, vsc=4 * A, nb=4, bs=16, Hkv=2, D=128, table=5 * A, mb=2,
             lens=6 * A, cu=7 * A, B=2, maxlen=20, ko=8 * A, vo=9 * A, rows=40, dtype=0, err=None,
             dev=0, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), pda.PDA_EINVAL), (dict(B=65536), pda.PDA_EINVAL), (dict(maxlen=-1), pda.PDA_EINVAL),
    (dict(maxlen=33), pda.PDA_EINVAL), (dict(rows=-1), pda.PDA_EINVAL), (dict(dtype=3), pda.PDA_EINVAL),
    (dict(D=80), pda.PDA_EUNSUPPORTED), (dict(bs=48), pda.PDA_EUNSUPPORTED), (dict(ko=None), pda.PDA_EINVAL),
    (dict(lens=None), pda.PDA_EINVAL), (dict(vo=9 * A + 8), pda.PDA_EINVAL), (dict(cu=7 * A + 4), pda.PDA_EINVAL),
    (dict(vo=8 * A), pda.PDA_EALIAS), (dict(ko=A), pda.PDA_EALIAS), (dict(ko=5 * A), pda.PDA_EALIAS),
    (dict(dev=-1), pda.PDA_EINVAL), (dict(B=0), pda.PDA_OK), (dict(maxlen=0), pda.PDA_OK),
    (dict(Hkv=8192), pda.PDA_EUNSUPPORTED), (dict(Hkv=0), pda.PDA_EINVAL), (dict(nb=0), pda.PDA_EINVAL),
])
def test_gather_refusals_before_cuda(lib, kw, status):
    assert lib.paged_decode_attn_gather_kv_fp8(*gather_args(**kw)) == status


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.float8_e4m3fn)
    sc = torch.ones(4, 2)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cu = torch.tensor([0, 1])
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pda.append_kv_fp8(k, k, kc, kc, sc, sc, table, lens, cu)
    with pytest.raises(ValueError):
        pda.gather_kv_fp8(kc, kc, sc, sc, table, lens)
    with pytest.raises(ValueError):
        pda.gather_kv_fp8(kc, kc, sc[:3], sc, table, lens)
    with pytest.raises(ValueError):
        pda.gather_kv_fp8(kc.to(torch.float32), kc, sc, sc, table, lens)
    assert ctypes.sizeof(ctypes.c_void_p) == 8
