"""Refusals of the 4-bit KV cache's entry points on the host: every argument that can be seen there is checked before any
HIP call (no GPU needed)."""
import ctypes as C
import os

import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

NULL, ARG, SHAPE, UNSUP, ALIGN = -1, -2, -3, -4, -6
P = [0x100000 * k for k in range(1, 12)]  # fake aligned device addresses, never used


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libfp4q.so not built")
    return B.lib()


def spec(**kw):
    s = B.make_spec(kw.pop("format", B.FP4Q_NVFP4), global_scale_given=True)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def cache(**kw):
    c = B.fp4q_kv_cache(*P[:6], 10, 2, 16, 128, 0, 2048, 1024, 64, 256, 128, 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def call(**kw):
    a = B.fp4q_attention(P[6], 1024, 128, P[7], 1024, 128, None, None, P[8], P[9], 8, 4, 8, 4, 1, 100, 8,
                         B.FP4Q_BF16, 1, 0, 0.1, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend(L, s=None, c=None, a=None, ws=None, n=0):
    return L.fp4q_attend(C.byref(s or spec()), C.byref(c or cache()), C.byref(a or call()), ws, n, None)


def write(L, s=None, c=None, k=P[6], v=P[7], dtype=B.FP4Q_BF16, tokens=4, st=(256, 128, 256, 128), slots=P[8]):
    return L.fp4q_kv_write(C.byref(s or spec()), C.byref(c or cache()), k, v, dtype, tokens, *st, slots, None)


def read(L, s=None, c=None, slots=P[6], tokens=4, k=P[7], v=P[8], dtype=B.FP4Q_F32):
    return L.fp4q_kv_read(C.byref(s or spec()), C.byref(c or cache()), slots, tokens, k, v, dtype, None)


BAD_CACHE = [(NULL, dict(k_codes=None)), (NULL, dict(v_scales=None)), (NULL, dict(k_global=None)),
             (ARG, dict(reserved=1)), (SHAPE, dict(num_pages=-1)), (SHAPE, dict(kv_heads=0)), (SHAPE, dict(page_size=0)),
             (UNSUP, dict(head_dim=96)), (UNSUP, dict(head_dim=512)), (SHAPE, dict(code_page=-16)),
             (SHAPE, dict(scale_token=-4)), (SHAPE, dict(code_token=1 << 21)), (SHAPE, dict(code_head=1 << 60)),
             (SHAPE, dict(num_pages=1 << 60)), (ALIGN, dict(k_codes=P[0] + 8)), (ALIGN, dict(v_scales=P[4] + 2)),
             (ALIGN, dict(code_token=72)), (ALIGN, dict(scale_head=130)), (ALIGN, dict(v_global=P[5] + 1))]
BAD_SPEC = [(ARG, dict(format=9)), (UNSUP, dict(format=B.FP4Q_IF4)), (UNSUP, dict(format=B.FP4Q_IF6)),
            (UNSUP, dict(block=32)), (ARG, dict(rotate=32)), (ARG, dict(rotate=8))]


@pytest.mark.parametrize("want,change", BAD_CACHE)
def test_bad_caches(L, want, change):
    for f in (write, read, attend):
        assert f(L, c=cache(**change)) == want


@pytest.mark.parametrize("want,change", BAD_SPEC)
def test_bad_specs(L, want, change):
    for f in (write, read, attend):
        assert f(L, s=spec(**change)) == want


def test_null_structs(L):
    s, c, a = spec(), cache(), call()
    assert L.fp4q_attend(None, C.byref(c), C.byref(a), None, 0, None) == NULL
    assert L.fp4q_attend(C.byref(s), None, C.byref(a), None, 0, None) == NULL
    assert L.fp4q_attend(C.byref(s), C.byref(c), None, None, 0, None) == NULL
    assert L.fp4q_attend_workspace_bytes(None, C.byref(c), C.byref(a)) == 0


def test_bad_writes(L):
    assert write(L, s=spec(scale_rule=7)) == ARG
    assert write(L, s=spec(objective=B.FP4Q_OBJ_WMSE)) == UNSUP
    assert write(L, s=spec(objective=5)) == ARG
    assert write(L, s=spec(global_scale_given=0)) == ARG
    assert write(L, s=spec(scale_rule=B.FP4Q_SCALE_SWEEP, sweep_lo=3, sweep_hi=2)) == ARG
    assert write(L, s=spec(scale_rule=B.FP4Q_SCALE_SWEEP, sweep_lo=-127)) == ARG
    mx = cache(scale_token=4, scale_head=64, scale_page=128)
    assert write(L, s=spec(format=B.FP4Q_MXFP4, scale_rule=B.FP4Q_SCALE_FOUR_OVER_SIX), c=mx) == UNSUP
    assert write(L, dtype=2) == ARG
    assert write(L, tokens=-1) == SHAPE
    assert write(L, tokens=1 << 62) == SHAPE
    assert write(L, st=(-8, 128, 256, 128)) == SHAPE
    assert write(L, k=None) == NULL and write(L, slots=None) == NULL
    assert write(L, k=P[6] + 8) == ALIGN and write(L, st=(256, 100, 256, 128)) == ALIGN
    assert write(L, slots=P[8] + 4) == ALIGN
    assert write(L, tokens=0, k=None, v=None, slots=None) == 0


def test_bad_reads(L):
    assert read(L, dtype=-1) == ARG
    assert read(L, tokens=-1) == SHAPE
    assert read(L, k=None) == NULL
    assert read(L, v=P[8] + 8) == ALIGN
    assert read(L, tokens=0, k=None, v=None, slots=None) == 0


@pytest.mark.parametrize("want,change", [
    (ARG, dict(dtype=3)), (ARG, dict(causal=2)), (ARG, dict(window=-1)), (ARG, dict(causal=0, window=4)),
    (ARG, dict(reserved=1)), (ARG, dict(scale=float("inf"))), (ARG, dict(scale=float("nan"))),
    (SHAPE, dict(batch=-1)), (SHAPE, dict(total_q=-4)), (SHAPE, dict(max_q=-1)), (SHAPE, dict(max_kv=-1)),
    (SHAPE, dict(q_heads=7)), (SHAPE, dict(q_heads=0)), (SHAPE, dict(table_len=-1)), (SHAPE, dict(table_stride=3)),
    (SHAPE, dict(q_row_stride=-8)), (SHAPE, dict(total_q=5)), (SHAPE, dict(total_q=1 << 60, q_starts=P[10])),
    (SHAPE, dict(max_q=(1 << 31) - 1, q_starts=P[10])), (SHAPE, dict(max_kv=(1 << 31) - 1)),
    (NULL, dict(q=None)), (NULL, dict(out=None)), (NULL, dict(kv_lens=None)),
    (ALIGN, dict(q=P[6] + 8)), (ALIGN, dict(out_head_stride=129)), (ALIGN, dict(lse=P[10] + 2)),
    (ALIGN, dict(kv_lens=P[8] + 1)), (ALIGN, dict(block_table=P[9] + 2))])
def test_bad_attention(L, want, change):
    assert attend(L, a=call(**change)) == want
    assert L.fp4q_attend_workspace_bytes(C.byref(spec()), C.byref(cache()), C.byref(call(**change))) == 0


def test_page_size_of_a_table(L):
    assert attend(L, c=cache(page_size=24)) == UNSUP


def test_empty_attention(L):
    assert attend(L, a=call(total_q=0, batch=0, q=None, out=None, kv_lens=None)) == 0
    assert attend(L, a=call(total_q=0, max_q=0, q=None, out=None, kv_lens=None)) == 0


def test_workspace(L):
    a = call(max_kv=5000, table_len=400, table_stride=400)
    n = L.fp4q_attend_workspace_bytes(C.byref(spec()), C.byref(cache()), C.byref(a))
    assert n > 0
    assert attend(L, a=a) == NULL
    assert attend(L, a=a, ws=P[10], n=n - 1) == ARG
    assert attend(L, a=a, ws=P[10] + 128, n=n) == ALIGN


def host_cache(fmt=B.FP4Q_NVFP4, **kw):
    blk = 32 if fmt == B.FP4Q_MXFP4 else 16
    t = dict(k_codes=torch.zeros(4, 2, 16, 64, dtype=torch.uint8), k_scales=torch.zeros(4, 2, 16, 128 // blk, dtype=torch.uint8),
             k_global=torch.ones(1), v_codes=torch.zeros(4, 2, 16, 64, dtype=torch.uint8),
             v_scales=torch.zeros(4, 2, 16, 128 // blk, dtype=torch.uint8), v_global=torch.ones(1))
    t.update(kw)
    return B.KvCache(**t, format=fmt, require_cuda=False)


def test_binding_refuses_caches():
    host_cache()
    host_cache(B.FP4Q_MXFP4, k_global=None, v_global=None)
    u8 = torch.uint8
    for kw in (dict(k_global=None), dict(k_codes=torch.zeros(4, 2, 16, 64)), dict(k_codes=torch.zeros(4, 2, 64, dtype=u8)),
               dict(v_codes=torch.zeros(4, 2, 15, 64, dtype=u8)), dict(k_scales=torch.zeros(4, 2, 16, 4, dtype=u8)),
               dict(v_global=torch.ones(1, dtype=torch.float64)),
               dict(v_codes=torch.zeros(4, 16, 2, 64, dtype=u8).transpose(1, 2)),
               dict(v_codes=torch.zeros(4, 2, 64, 16, dtype=u8).transpose(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            host_cache(**kw)
    with pytest.raises(ValueError):
        host_cache(B.FP4Q_IF4)
    with pytest.raises(ValueError):  # a host tensor where a device's is expected
        c = host_cache()
        B.KvCache(*c.tensors)
    with pytest.raises(ValueError):
        B.alloc_kv_cache(1, 1, 16, 64, device="cpu")


def test_binding_refuses_calls():
    c = host_cache()
    x = torch.zeros(3, 2, 128)
    slots = torch.zeros(3, dtype=torch.int64)
    for k, v, s in ((x[:2], x, slots), (x.double(), x.double(), slots), (x, x.bfloat16(), slots), (x, x, slots.int()),
                    (x[:, :1], x[:, :1], slots), (torch.zeros(3, 128, 2).transpose(1, 2), x, slots), (x, x, slots[None])):
        with pytest.raises((ValueError, TypeError)):
            B.kv_write(c, k, v, s)
    with pytest.raises((ValueError, TypeError)):
        B.kv_read(c, slots, dtype=torch.float16)
    q = torch.zeros(4, 8, 128)
    lens = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros(4, 2, dtype=torch.int32)
    starts = torch.zeros(5, dtype=torch.int32)
    B.attend_workspace_bytes(c, q, lens, block_table=table)
    for kw in (dict(q=q[0]), dict(q=q[:, :3]), dict(q=q.half()), dict(q=q[:3]), dict(kv_lens=lens.long()),
               dict(block_table=table[:3]), dict(block_table=table.long()), dict(q_starts=starts[:4]), dict(max_q=2),
               dict(q=torch.zeros(4, 128, 8).transpose(1, 2)), dict(block_table=torch.zeros(2, 4, dtype=torch.int32).T)):
        args = dict(q=q, kv_lens=lens, block_table=table)
        args.update(kw)
        with pytest.raises((ValueError, TypeError)):
            B.attend_workspace_bytes(c, **args)


def test_binding_refuses_sizes_past_31_bits():
    c = host_cache()
    q = torch.zeros(4, 8, 128)
    lens = torch.zeros(4, dtype=torch.int32)
    starts = torch.zeros(5, dtype=torch.int32)
    for kw in (dict(max_kv=(1 << 32) + 16), dict(max_kv=1 << 31), dict(max_kv=-1), dict(window=1 << 32),
               dict(window=-1), dict(max_q=(1 << 32) + 1, q_starts=starts), dict(max_q=-1, q_starts=starts)):
        with pytest.raises(ValueError):
            B.attend_workspace_bytes(c, q, lens, **kw)
    # the default bound, what 2^27 pages of 16 tokens hold, does not fit
    wide = torch.empty(1, 1 << 27, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_kv"):
        B.attend_workspace_bytes(c, q, lens[:1], block_table=wide)
    B.attend_workspace_bytes(c, q, lens[:1], block_table=wide, max_kv=4096)
