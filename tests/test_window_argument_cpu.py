"""What run takes as window; no GPU: the library's call is recorded in its place."""
import numpy as np
import pytest
import torch

from paged_gqa_decode_attention_gb300 import PagedDecodeAttention, _binding


@pytest.fixture
def call(monkeypatch):
    class Recorder:
        def paged_decode_attn_run_scored(self, *args):
            self.window = args[12]
            return 0
    a = PagedDecodeAttention.__new__(PagedDecodeAttention)
    a.lib, a.handle, a.device, a.dtype, a.kv_fp8 = Recorder(), None, 0, torch.bfloat16, False
    a._geometry = (4, 2, 16, 64)
    monkeypatch.setattr(_binding, "_pointers", lambda dev, named: [1 << 20] * len(named))
    q, cache = torch.zeros(2, 4, 64).bfloat16(), torch.zeros(3, 16, 2, 64).bfloat16()

    def run(window):
        a.run(q, cache, cache, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), window=window,
              stream=0)
        return a.lib.window
    return run


@pytest.mark.parametrize("window,passed", [(1, 1), (1024, 1024), (np.int64(77), 77), (2 ** 31 - 1, 2 ** 31 - 1),
                                           (2 ** 31, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                           (10 ** 12, 2 ** 31 - 1), (-1, -1), (-2 ** 32, -1), (-2 ** 31 - 7, -1)])
def test_integers_reach_the_library_without_losing_bits(call, window, passed):
    assert call(window) == passed


@pytest.mark.parametrize("window", [0.5, 2.5, 100.0, float("nan"), "9"])
def test_anything_else_is_refused(call, window):
    with pytest.raises(ValueError, match="window"):
        call(window)
