"""CPU: caches that rotary positions and append cannot write to."""
import os

import pytest

import block_scaled_fp8_fp8blk_amd as fb
from test_attention_refusals import P, S, append, attn


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fb.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fb.load()


def test_keys_and_values_in_the_same_rows(lib):
    """Both would be written there, and either left; attention only reads them."""
    assert append(lib, c=dict(v=P)) == fb.ERR_ARG
    assert append(lib, c=dict(k=P + S, v=P + S)) == fb.ERR_ARG
    assert attn(lib, c=dict(v=P), wsb=0, batch=dict(max_len=100000)) == fb.ERR_WORKSPACE  # past the checks of its arguments
