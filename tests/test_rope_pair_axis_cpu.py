"""What rope_axes_kv_write takes as pair_axis; no GPU: the library's call is recorded in its place."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_attention_gb300 as pda
from paged_gqa_decode_attention_gb300 import _binding

AXES = [0, 1, 2, 0, 1, 2, 1, 1]


class Recorder:
    def __init__(self):
        self.args = None

    def paged_decode_attn_rope_axes_kv_write(self, *args):
        self.args = args
        return 0


@pytest.fixture
def call(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(_binding, "_lib", lib)
    monkeypatch.setattr(_binding, "_cuda_device", lambda t: 0)
    monkeypatch.setattr(_binding, "_rows16", lambda *a: (1 << 20, 128))
    monkeypatch.setattr(_binding, "_pointers", lambda dev, named: [1 << 20] * len(named))
    q, k = torch.zeros(4, 8, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16()
    cache = torch.zeros(2, 16, 2, 64).bfloat16()

    def run(axes, rot=16):
        pda.rope_axes_kv_write(q, k, k, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64),
                               torch.zeros(9, rot), cache, cache.clone(), axes, stream=0)
        return lib.args[8]
    return run


@pytest.mark.parametrize("axes", [AXES, tuple(AXES), bytes(AXES), iter(AXES), np.array(AXES), np.array(AXES, np.int16),
                                  np.array(AXES, np.uint8), torch.tensor(AXES), torch.tensor(AXES, dtype=torch.uint8)])
def test_integers_of_any_kind(call, axes):
    assert call(axes) == bytes(AXES)


def test_no_pairs(call):
    assert call([], 0) == b""


# a number is no list of zeros, and an array's memory is not its values
@pytest.mark.parametrize("axes", [8, np.int64(8), True, None, "01201211", [0.0] * 8, np.zeros(8), AXES[:7], AXES + [0],
                                  [-1] * 8, [256] * 8, np.array([0x0201000102010001]), torch.tensor(8)])
def test_anything_else_is_refused(call, axes):
    with pytest.raises(ValueError):
        call(axes)
