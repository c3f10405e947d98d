"""Block counts whose product with the block size does not fit 64 bits are refused
before any CUDA call, as those just past 2^31 slots are."""
import pytest

import paged_gqa_decode_attention_gb300 as pda
from paged_gqa_decode_attention_gb300 import build as pda_build
from test_fp8_cache_cpu import A, append_args, gather_args, rope_args

COUNTS = [1 << 27, 1 << 59, 1 << 60, (1 << 60) + 1, (1 << 62) + 3]  # blocks of 16 and 32


@pytest.fixture(scope="module")
def lib():
    pda_build.build()
    return pda.load_library()


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("nb", COUNTS)
def test_refused(lib, nb, bs):
    assert lib.paged_decode_attn_append_kv_fp8(*append_args(nb=nb, bs=bs)) == pda.PDA_EINVAL
    assert lib.paged_decode_attn_rope_append_kv_fp8(*rope_args(nb=nb, bs=bs)) == pda.PDA_EINVAL
    assert lib.paged_decode_attn_gather_kv_fp8(*gather_args(nb=nb, bs=bs)) == pda.PDA_EINVAL
    assert lib.paged_decode_attn_run_noalloc(A, 2 * A, 3 * A, 4 * A, 5 * A, 1, 32, 8, 128, bs, 0, 4, nb, 0.1,
                                             6 * A, 0, 0, None) == pda.PDA_EINVAL
    message = lib.paged_decode_attn_last_error()
    assert b"num_blocks" in message, message
