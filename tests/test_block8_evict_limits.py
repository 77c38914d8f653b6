"""Sizes at the end of 32 bits that the block-scaled cache's, the 4-bit cache's and the eviction's entry
points refuse, without a GPU: the C ABI's host checks answer before any pointer is used."""
import ctypes

import pytest

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build

P = ctypes.c_void_p(16 * 1024)      # aligned, never dereferenced
UNSUPPORTED = 6


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


@pytest.mark.parametrize("W,keep", [(2 ** 31 - 1, 8), (64, 2 ** 31 - 1), (2 ** 31 - 1024, 8), (8, 2 ** 31 - 1024)])
def test_select_tokens_rows_that_a_step_of_its_loops_takes_past_32_bits(lib, W, keep):
    """A CTA's threads walk a row 1024 places at a time, in 32 bits."""
    assert lib.pa_select_tokens(P, 1, W, P, P, 1, 1, keep, 0, 0, P, P, P, None) == UNSUPPORTED


@pytest.mark.parametrize("fmt,Hkv", [("int8_block", 1 << 20), ("fp8_block", 1 << 22), ("int4", 1 << 21)])
def test_decode_blocks_of_4_gib(lib, fmt, Hkv):
    """A block's bytes over all KV heads, by which a block is found, are counted in 32 bits."""
    assert getattr(lib, "pa_decode_" + fmt)(P, P, P, P, P, P, 1, P, 8, 1, Hkv, Hkv, 128, 32, 2, 0.1, 0, P, P, 1 << 40,
                                            None) == UNSUPPORTED
