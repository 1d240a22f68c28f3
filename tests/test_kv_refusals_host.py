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


@pytest.mark.parametrize("change", [
    dict(code_token=0), dict(code_token=32), dict(code_head=512), dict(code_page=1024), dict(code_head=0, code_page=0),
    dict(scale_token=4), dict(scale_head=64), dict(scale_page=252), dict(v_codes=P[0]), dict(v_scales=P[1])])
def test_written_caches_whose_rows_share_bytes(L, change):
    """Expanded and overlapping caches cannot be written."""
    assert write(L, c=cache(**change)) == SHAPE
    assert read(L, c=cache(**change), tokens=0) == 0  # but read


@pytest.mark.parametrize("change", [
    dict(), dict(code_head=64, code_token=128), dict(scale_head=8, scale_token=16), dict(code_page=4096),
    dict(kv_heads=1, code_head=0), dict(num_pages=1, code_page=0), dict(page_size=1, code_token=0, code_head=64),
    dict(num_pages=0, code_token=0)])
def test_written_caches_whose_rows_lie_apart(L, change):
    """Any order of the dimensions, wider pages, and strides of dimensions that have one entry."""
    assert write(L, c=cache(**change), tokens=0) == 0


@pytest.mark.parametrize("change", [dict(out_row_stride=0), dict(out_head_stride=0), dict(out_head_stride=64),
                                    dict(out_row_stride=1016), dict(out_row_stride=128, out_head_stride=128)])
def test_outputs_whose_rows_share_elements(L, change):
    assert attend(L, a=call(**change)) == SHAPE
    assert L.fp4q_attend_workspace_bytes(C.byref(B.make_spec(global_scale_given=True)), C.byref(cache()),
                                         C.byref(call(**change))) == 0


def test_outputs_whose_rows_lie_apart(L):
    """Heads outside rows, wider rows, single rows and heads: refused only for the workspace that is missing."""
    big = dict(max_kv=5000, table_len=400, table_stride=400)
    for change in (dict(), dict(out_row_stride=128, out_head_stride=512), dict(out_row_stride=4096),
                   dict(q_heads=2, out_head_stride=128, out_row_stride=256)):
        assert attend(L, a=call(**big, **change)) == -1, change
    one = dict(batch=1, total_q=1, out_row_stride=0)
    assert attend(L, a=call(**big, **one)) == -1


def test_workspace_of_expanded_queries():
    """Queries may be expanded (only outputs may not); the workspace is that of their copies."""
    t = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, 8, dtype=torch.uint8), torch.ones(1)]
    c = B.KvCache(*t, *[x.clone() for x in t], require_cuda=False)
    lens, table = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 400, dtype=torch.int32)
    q = torch.zeros(1, 1, 128).expand(4, 8, 128)
    need = B.attend_workspace_bytes(c, q, lens, block_table=table)
    assert need == B.attend_workspace_bytes(c, q.contiguous(), lens, block_table=table) > 0


def test_expanded_tensors():
    """Heads of one tensor expanded: a cache that can be read, not written."""
    code = [torch.zeros(4, 1, 16, 64, dtype=torch.uint8).expand(4, 2, 16, 64) for _ in range(2)]
    scale = [torch.zeros(4, 2, 16, 8, dtype=torch.uint8) for _ in range(2)]
    c = B.KvCache(code[0], scale[0], torch.ones(1), code[1], scale[1], torch.ones(1), require_cuda=False)
    c.struct.k_codes = P[0]  # the library sees aligned addresses
    c.struct.k_scales, c.struct.v_codes, c.struct.v_scales = P[1], P[3], P[4]
    assert write(B.lib(), s=c.spec, c=c.struct) == SHAPE
    assert read(B.lib(), s=c.spec, c=c.struct, tokens=0) == 0


def test_long_bounds_of_many_sequences_are_not_refused():
    """512 sequences of 32 heads under a bound of 131072 keys: 16384 pairs of up to 1024 steps each, in 16384 workgroups
    and one round more. Steps are counted in 31 bits, and only what goes past those is refused."""
    L = B.lib()
    s = B.make_spec(global_scale_given=True)
    c = cache(kv_heads=32, code_page=32 * 1024, scale_page=32 * 128)
    for max_kv, fits in ((131072, True), (1 << 23, True), (1 << 25, False)):
        a = call(batch=512, total_q=512, max_q=1, q_heads=32, out_row_stride=4096, q_row_stride=4096, max_kv=max_kv)
        assert (L.fp4q_attend_workspace_bytes(C.byref(s), C.byref(c), C.byref(a)) > 0) == fits, max_kv
        assert attend(L, s=s, c=c, a=a) == (-1 if fits else SHAPE), max_kv  # -1: the workspace is missing
