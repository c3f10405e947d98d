"""The shared-prefix, scored and several-axes calls without a GPU: refusals before any CUDA call,
and the assignment of rotary pairs to axes."""
import ctypes

import pytest
import torch

import paged_gqa_decode_attention_gb300 as pda
from paged_gqa_decode_attention_gb300 import build as pda_build


@pytest.fixture(scope="module")
def lib():
    pda_build.build()
    return pda.load_library()


def test_pair_axes():
    assert pda.rope_pair_axes((2, 3, 1)) == [0, 0, 1, 1, 1, 2]
    assert pda.rope_pair_axes((3, 2, 2), interleaved=True) == [0, 1, 2, 0, 1, 2, 0]
    assert pda.rope_pair_axes((1, 4), interleaved=True) == [0, 1, 1, 1, 1]
    assert pda.rope_pair_axes(()) == [] == pda.rope_pair_axes((), True)


def test_null_handle_is_refused(lib):
    z = [None] * 5
    assert lib.paged_decode_attn_run_scored(None, *z, 1, 1, 1, 1.0, 0.0, None, 0, None, None) == pda.PDA_EINVAL
    assert lib.paged_decode_attn_run_shared_prefix(None, *z, 1, 1, 1, None, None, 1, 1.0, 0.0, None, None,
                                                   None) == pda.PDA_EINVAL
    assert b"handle" in lib.paged_decode_attn_last_error()


@pytest.mark.parametrize("axes,pairs,status", [(0, bytes(32), pda.PDA_EINVAL), (5, bytes(32), pda.PDA_EINVAL),
                                               (3, bytes([0, 1, 2, 3] * 8), pda.PDA_EINVAL),
                                               (3, None, pda.PDA_EINVAL)])
def test_axes_are_checked_first(lib, axes, pairs, status):
    p = ctypes.c_void_p(1 << 20)  # never dereferenced
    got = lib.paged_decode_attn_rope_axes_kv_write(p, 0, p, 0, p, 0, p, axes, pairs, p, p, 100, 64, 1, 4, 8, 2,
                                                   64, pda.PDA_BF16, p, 0, p, p, 64, None, 0, None)
    assert got == status


def test_outputs_over_inputs_are_refused(lib):
    mb = 1 << 20
    at = [ctypes.c_void_p(mb * (i + 1)) for i in range(9)]
    q, k, v, pos, slots, cs, out, kc, vc = at

    def call(positions):
        return lib.paged_decode_attn_rope_axes_kv_write(q, 0, k, 0, v, 0, positions, 3, bytes(32), slots, cs, 100,
                                                        64, 1, 4, 8, 2, 64, pda.PDA_BF16, out, 0, kc, vc, 64, None,
                                                        0, None)

    # the third axis's positions reach into q_out
    assert call(ctypes.c_void_p(mb * 7 - 40)) == pda.PDA_EALIAS


def test_cpu_tensors_are_refused():
    q, k = torch.zeros(4, 8, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16()
    cache = torch.zeros(2, 16, 2, 64).bfloat16()
    with pytest.raises(ValueError, match="CUDA"):
        pda.rope_axes_kv_write(q, k, k, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64),
                               torch.zeros(9, 64), cache, cache.clone(), [0] * 32)
