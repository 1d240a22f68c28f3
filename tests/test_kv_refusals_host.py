"""Refusals of the 4-bit KV cache's entry points on the host: offsets past 63 bits and rows that would be written twice
at once (no GPU needed; nothing reaches the HIP runtime)."""
import ctypes as C
import os

import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from test_kv_host import P, attend, cache, call, read, write

SHAPE = -3


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libfp4q.so not built")
    return B.lib()


@pytest.mark.parametrize("change", [dict(code_head=1 << 46), dict(scale_head=1 << 46)])
def test_head_offsets_of_a_cache(L, change):
    c = cache(kv_heads=1 << 20, **change)
    assert write(L, c=c) == SHAPE and read(L, c=c) == SHAPE
    assert attend(L, c=c, a=call(q_heads=1 << 20)) == SHAPE


def test_head_offsets_of_rows(L):
    c = cache(kv_heads=1 << 18)
    for st in ((256, 1 << 46, 256, 128), (256, 128, 256, 1 << 46)):
        assert write(L, c=c, st=st) == SHAPE
    for change in (dict(q_head_stride=1 << 46), dict(out_head_stride=1 << 46)):
        assert attend(L, a=call(q_heads=1 << 18, **change)) == SHAPE
