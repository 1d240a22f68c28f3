"""Refusals of the products with 4-bit weights and of the cache's append on the host: every argument that can be seen there is
checked before any HIP call (no GPU needed)."""
import ctypes as C
import os

import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from test_kv_host import cache

NULL, ARG, SHAPE, UNSUP, ALIGN = -1, -2, -3, -4, -6
P = [0x100000 * k for k in range(1, 14)]  # fake aligned device addresses, never used


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libfp4q.so not built")
    return B.lib()


def spec(**kw):
    s = B.make_spec(kw.pop("format", B.FP4Q_NVFP4))
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def weight(**kw):
    w = B.fp4q_weight(P[0], P[1], P[2], 100, 256)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def matmul(L, s=None, w=None, x=P[3], dtype=B.FP4Q_BF16, tokens=4, xs=256, y=P[4], ys=100, ws=None, n=0):
    return L.fp4q_matmul(C.byref(s or spec()), C.byref(w or weight()), x, dtype, tokens, xs, y, ys, ws, n, None)


def gated(L, s=None, g=None, u=None, act=0, x=P[3], dtype=B.FP4Q_BF16, tokens=4, xs=256, y=P[4], ys=100, ws=None, n=0):
    return L.fp4q_gated(C.byref(s or spec()), C.byref(g or weight()), C.byref(u or weight()), act, x, dtype, tokens, xs, y, ys,
                        ws, n, None)


BAD_SPEC = [(ARG, dict(format=9)), (ARG, dict(format=-1)), (UNSUP, dict(format=B.FP4Q_IF4)), (UNSUP, dict(format=B.FP4Q_IF6)),
            (UNSUP, dict(block=32)), (ARG, dict(rotate=8)), (ARG, dict(rotate=32))]
BAD_WEIGHT = [(NULL, dict(codes=None)), (NULL, dict(scales=None)), (NULL, dict(global_scale=None)), (SHAPE, dict(rows=-1)),
              (SHAPE, dict(cols=-16)), (SHAPE, dict(cols=250)), (SHAPE, dict(cols=(1 << 22) + 16)), (SHAPE, dict(rows=1 << 37)),
              (ALIGN, dict(codes=P[0] + 4)), (ALIGN, dict(global_scale=P[2] + 2))]
BAD_CALL = [(ARG, dict(dtype=2)), (SHAPE, dict(tokens=-1)), (SHAPE, dict(tokens=1 << 31)), (SHAPE, dict(xs=-8)),
            (SHAPE, dict(xs=1 << 40)), (SHAPE, dict(ys=-1)), (SHAPE, dict(ys=99)), (SHAPE, dict(ys=1 << 60)), (NULL, dict(x=None)),
            (NULL, dict(y=None)), (ALIGN, dict(x=P[3] + 8)), (ALIGN, dict(xs=260)), (ALIGN, dict(y=P[4] + 1)),
            (ALIGN, dict(dtype=B.FP4Q_F32, xs=258)), (ALIGN, dict(dtype=B.FP4Q_F32, y=P[4] + 2))]


@pytest.mark.parametrize("status,change", BAD_SPEC)
def test_specs(L, status, change):
    assert matmul(L, s=spec(**change)) == status and gated(L, s=spec(**change)) == status
    assert L.fp4q_matmul_workspace_bytes(C.byref(spec(**change)), C.byref(weight()), 300, B.FP4Q_F32) == 0


@pytest.mark.parametrize("status,change", BAD_WEIGHT)
def test_weights(L, status, change):
    w = weight(**change)
    assert matmul(L, w=w) == status and gated(L, g=w) == status and gated(L, u=w) == status
    assert L.fp4q_matmul_workspace_bytes(C.byref(spec()), C.byref(w), 300, B.FP4Q_F32) == 0
    assert L.fp4q_gated_workspace_bytes(C.byref(spec()), C.byref(w), 300, B.FP4Q_F32) == 0


@pytest.mark.parametrize("status,change", BAD_CALL)
def test_calls(L, status, change):
    assert matmul(L, **change) == status and gated(L, **change) == status


def test_mxfp4_weights(L):
    mx = spec(format=B.FP4Q_MXFP4)
    assert matmul(L, s=mx, w=weight(codes=P[0] + 8)) == ALIGN
    assert matmul(L, s=mx, w=weight(cols=272)) == SHAPE
    assert matmul(L, s=mx, w=weight(global_scale=None), tokens=0) == 0


def test_pairs_and_activations(L):
    assert gated(L, u=weight(rows=101)) == SHAPE and gated(L, u=weight(cols=272), xs=272) == SHAPE
    for act in (-1, 3):
        assert gated(L, act=act) == ARG


def test_workspaces(L):
    """Where a call needs one it says how much, and refuses none, a short and an unaligned one."""
    need = L.fp4q_matmul_workspace_bytes(C.byref(spec()), C.byref(weight()), 300, B.FP4Q_F32)
    assert need >= 300 * 256 * 2 * 2  # two parts of x at least
    big = dict(tokens=300, dtype=B.FP4Q_F32)
    assert matmul(L, **big) == NULL
    assert matmul(L, ws=P[5], n=need - 1, **big) == ARG
    assert matmul(L, ws=P[5] + 64, n=need, **big) == ALIGN
    assert L.fp4q_matmul_workspace_bytes(C.byref(spec()), C.byref(weight()), 1, B.FP4Q_BF16) == 0
    for tokens in (0, -3):
        assert L.fp4q_matmul_workspace_bytes(C.byref(spec()), C.byref(weight()), tokens, B.FP4Q_F32) == 0
    assert L.fp4q_matmul_workspace_bytes(C.byref(spec()), C.byref(weight()), 300, 7) == 0


def test_nulls(L):
    assert L.fp4q_matmul(None, C.byref(weight()), P[3], 1, 4, 256, P[4], 100, None, 0, None) == NULL
    assert L.fp4q_matmul(C.byref(spec()), None, P[3], 1, 4, 256, P[4], 100, None, 0, None) == NULL
    assert L.fp4q_gated(C.byref(spec()), C.byref(weight()), None, 0, P[3], 1, 4, 256, P[4], 100, None, 0, None) == NULL
    assert L.fp4q_matmul_workspace_bytes(None, None, 4, 1) == 0


def test_empty_calls(L):
    assert matmul(L, tokens=0, x=None, y=None) == 0
    assert matmul(L, w=weight(rows=0, codes=None, scales=None, global_scale=None), ys=0, y=None) == 0


# ---- the plan: what any size asks for stays within what a launch and 32-bit offsets hold -----------------------------

@pytest.mark.parametrize("fmt", [B.FP4Q_NVFP4, B.FP4Q_MXFP4])
@pytest.mark.parametrize("dtype", [B.FP4Q_BF16, B.FP4Q_F32])
def test_workspace_grows_as_the_parts_and_partial_sums(L, fmt, dtype):
    """Parts of x, exponents and whole tiles of partial sums are all that a call asks for."""
    for rotate in (0, 32 if fmt == B.FP4Q_MXFP4 else 16):
        s = spec(format=fmt, rotate=rotate)
        exact = dtype == B.FP4Q_BF16 and not rotate
        for tokens in (1, 4, 5, 16, 17, 33, 64, 65, 509, 8192):
            for n, k in ((1, 32), (100, 256), (4096, 4096), (14336, 4096), (33, 14336)):
                got = L.fp4q_matmul_workspace_bytes(C.byref(s), C.byref(weight(rows=n, cols=k)), tokens, dtype)
                parts = 0 if exact else (3 if dtype == B.FP4Q_F32 else 2)
                tile = 32 if tokens <= 32 else (64 if tokens <= 64 else 128)
                rows = -(-tokens // tile) * tile
                most = parts * tokens * k * 2 + tokens * 4 + 1024 + max(4 * 256 * tile, rows * 4) * 256 * 4 * 4
                assert 0 <= got <= most
                if tokens <= 2 or (exact and tokens <= 16):
                    assert got == 0


# ---- the cache's append -------------------------------------------------------------------------------------------------

def call(**kw):
    c = B.fp4q_append(q=P[6], q_row_stride=1024, q_head_stride=128, q_out=P[7], out_row_stride=1024, out_head_stride=128,
                      k=P[8], k_token_stride=256, k_head_stride=128, v=P[9], v_token_stride=256, v_head_stride=128,
                      q_weight=P[10], k_weight=P[10], rope=P[11], rope_stride=64, rope_rows=100, positions=P[12], slots=P[5],
                      tokens=4, q_heads=8, rope_dim=64, interleaved=0, dtype=B.FP4Q_BF16, eps=1e-6, reserved=0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(L, s=None, c=None, a=None):
    s = s or B.make_spec(global_scale_given=True)
    return L.fp4q_kv_append(C.byref(s), C.byref(c or cache()), C.byref(a or call()), None)


BAD_APPEND = [(ARG, dict(dtype=3)), (ARG, dict(interleaved=2)), (ARG, dict(reserved=1)), (ARG, dict(eps=0.0)),
              (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))), (ARG, dict(eps=float("inf"))), (SHAPE, dict(tokens=-1)),
              (SHAPE, dict(q_heads=-1)), (SHAPE, dict(rope_dim=-16)), (SHAPE, dict(rope_dim=24)), (SHAPE, dict(rope_dim=144)),
              (SHAPE, dict(rope_rows=-1)), (SHAPE, dict(rope_stride=-4)), (SHAPE, dict(rope_stride=1 << 50)),
              (SHAPE, dict(rope_rows=1 << 60)), (SHAPE, dict(q_row_stride=-8)), (SHAPE, dict(k_head_stride=1 << 60)),
              (SHAPE, dict(tokens=1 << 58)), (SHAPE, dict(q_heads=1 << 30)), (NULL, dict(q=None)), (NULL, dict(q_out=None)),
              (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(slots=None)), (NULL, dict(positions=None)),
              (NULL, dict(rope=None)), (ALIGN, dict(q=P[6] + 8)), (ALIGN, dict(q_out=P[7] + 2)), (ALIGN, dict(k_token_stride=260)),
              (ALIGN, dict(v=P[9] + 4)), (ALIGN, dict(rope=P[11] + 4)), (ALIGN, dict(rope_stride=66)), (ALIGN, dict(positions=P[12] + 4)),
              (ALIGN, dict(slots=P[5] + 4)), (ALIGN, dict(q_weight=P[10] + 4)), (ALIGN, dict(k_weight=P[10] + 8)),
              (SHAPE, dict(out_row_stride=0)), (SHAPE, dict(out_head_stride=64))]


@pytest.mark.parametrize("status,change", BAD_APPEND)
def test_appends(L, status, change):
    assert append(L, a=call(**change)) == status


def test_appends_in_place_take_one_layout(L):
    """q_out may be q where each row is overwritten by its own result alone."""
    for change in (dict(out_row_stride=2048), dict(q_row_stride=2048), dict(out_row_stride=128, out_head_stride=512)):
        assert append(L, a=call(q_out=P[6], **change)) == SHAPE
    assert append(L, a=call(q_out=P[6], tokens=0, out_row_stride=2048)) == 0


def test_appends_to_caches_that_cannot_be_written(L):
    for change in (dict(code_token=0), dict(scale_head=64), dict(v_codes=P[0])):
        assert append(L, c=cache(**change)) == SHAPE
    assert append(L, s=B.make_spec(B.FP4Q_IF4, global_scale_given=True)) == UNSUP
    assert append(L, s=B.make_spec(objective=B.FP4Q_OBJ_WMSE, global_scale_given=True)) == UNSUP
    assert append(L, s=B.make_spec(global_scale_given=False)) == ARG
    assert append(L, c=cache(reserved=1)) == ARG


def test_appends_without_work(L):
    """No tokens; what is not used is not looked at."""
    assert append(L, a=call(tokens=0, q=None, k=None, slots=None)) == 0
    assert append(L, a=call(tokens=0, rope_dim=0, rope=7, rope_stride=-3, rope_rows=-5, positions=None)) == 0
    assert append(L, a=call(tokens=0, q_heads=0, q=3, q_row_stride=-1, out_head_stride=5)) == 0
    assert append(L, a=call(tokens=0, q_weight=None, k_weight=None, eps=0.0)) == 0


# ---- the binding's own checks -----------------------------------------------------------------------------------------------

def host_weight(n=8, k=64, **kw):
    return B.QuantizedWeight(torch.zeros(n * k // 2, dtype=torch.uint8), torch.zeros(n * k // 16, dtype=torch.uint8),
                             torch.ones(1), n, k, require_cuda=False, **kw)


def test_binding_refuses_weights(L):
    c, s, g = torch.zeros(256, dtype=torch.uint8), torch.zeros(32, dtype=torch.uint8), torch.ones(1)
    for bad in (dict(codes=c[:255]), dict(scales=s[:31]), dict(global_scale=None), dict(codes=c.float()), dict(rows=-1),
                dict(cols=60), dict(cols=(1 << 22) + 16), dict(format=B.FP4Q_IF4), dict(rotate=32), dict(scales=s[::2])):
        a = dict(codes=c, scales=s, global_scale=g, rows=8, cols=64, require_cuda=False)
        a.update(bad)
        with pytest.raises(ValueError):
            B.QuantizedWeight(**a)
    with pytest.raises(TypeError):
        B.QuantizedWeight(None, s, g, 8, 64)
    with pytest.raises(ValueError):  # a host tensor
        B.QuantizedWeight(c, s, g, 8, 64)


def test_binding_refuses_rows(L):
    w = host_weight()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (x.half(), x[:, :48], x.t(), x.view(2, 2, 64)[:, :, :32], torch.zeros(4, 128, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError):
            B._product("fp4q_matmul", (w,), (), bad, None, None)
    for out in (torch.zeros(4, 9, dtype=torch.bfloat16), torch.zeros(4, 8), torch.zeros(5, 8, dtype=torch.bfloat16),
                torch.zeros(8, 4, dtype=torch.bfloat16).t()):
        with pytest.raises(ValueError):
            B._product("fp4q_matmul", (w,), (), x, out, None)
    with pytest.raises(TypeError):
        B._product("fp4q_matmul", (w,), (), None, None, None)
    with pytest.raises(ValueError):
        B.gated(w, host_weight(9), x)
    with pytest.raises(ValueError):
        B.gated(w, host_weight(rotate=16), x)


def test_binding_refuses_appends(L):
    c = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 16, 8, dtype=torch.uint8)
    cache_ = B.KvCache(c[0], c[1], torch.ones(1), c[0].clone(), c[1].clone(), torch.ones(1), require_cuda=False)
    k = torch.zeros(4, 2, 128)
    slots, pos = torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)
    table, w = torch.zeros(9, 64), torch.ones(128)
    good = dict(k=k, v=k, slots=slots, q=torch.zeros(4, 6, 128), positions=pos, rope=table, q_weight=w, k_weight=w)
    for bad in (dict(k=k[:3]), dict(v=k.bfloat16()), dict(slots=slots.int()), dict(q=torch.zeros(3, 6, 128)),
                dict(q=torch.zeros(4, 6, 64)), dict(q=torch.zeros(4, 6, 128).bfloat16()), dict(positions=None),
                dict(positions=pos[:3]), dict(positions=pos.int()), dict(rope=table.double()), dict(rope=table[:, :40]),
                dict(rope=torch.zeros(9, 144)), dict(rope=table[:, :0]), dict(rope=torch.zeros(64, 9).t()), dict(q_weight=w[:64]),
                dict(k_weight=w.bfloat16()), dict(out=torch.zeros(4, 5, 128)), dict(q=None, out=torch.zeros(4, 6, 128))):
        with pytest.raises(ValueError):
            B.kv_append(cache_, **{**good, **bad})
    for bad in (dict(q=3), dict(rope=3), dict(q_weight=3), dict(k=3)):
        with pytest.raises(TypeError):
            B.kv_append(cache_, **{**good, **bad})
