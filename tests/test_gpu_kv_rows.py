"""Writing tokens into the 4-bit KV cache and reading them back: every byte against the CPU oracle."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from oracle import ref
from kv_common import FMT, as_bf16, values

pytestmark = pytest.mark.gpu
RULES = {"absmax": (B.FP4Q_SCALE_ABSMAX, ref.ABSMAX), "sweep": (B.FP4Q_SCALE_SWEEP, ref.SWEEP),
         "foursix": (B.FP4Q_SCALE_FOUR_OVER_SIX, ref.FOUR_SIX)}


def host(x):
    return x.view(torch.int16).cpu().numpy().view(np.uint16) if x.dtype == torch.bfloat16 else x.cpu().numpy()


def write_and_check(rng, x, fmt, rule, rotate=False, window=None, page=16, S=(0.01, 0.02), strided=False, drop=()):
    """x: K and V, torch [T, H, D] on the host.  Writes them at random slots and compares the whole cache."""
    f, rf, block = FMT[fmt]
    T, H, D = x[0].shape
    pages = -(-T // page) + 2
    cache = B.alloc_kv_cache(pages, H, page, D, *S, format=f, scale_rule=RULES[rule][0], window=window,
                             rotate=block if rotate else 0)
    for t in (cache.tensors[0], cache.tensors[1], cache.tensors[3], cache.tensors[4]):
        t.fill_(0xA5)
    slots = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int64))
    given = slots.clone()
    for i, bad in drop:
        given[i] = bad if bad < 0 else pages * page + bad
    dev = []
    for t in x:
        t = t.cuda()
        if strided:  # heads outside tokens, in a wider allocation
            wide = torch.empty(H, T + 3, 2 * D, dtype=t.dtype, device="cuda")
            wide[:, :T, D:] = t.transpose(0, 1)
            t = wide[:, :T, D:].transpose(0, 1)
        dev.append(t)
    B.kv_write(cache, dev[0], dev[1], given.cuda())
    torch.cuda.synchronize()
    kept = np.ones(T, bool)
    for i, _ in drop:
        kept[i] = False
    at = slots.numpy()[kept]
    for side in range(2):
        rows = host(x[side].contiguous().reshape(T * H, D))
        want = ref.quantize(rows, fmt=rf, rule=RULES[rule][1], window=window, rotate=block if rotate else 0,
                            global_scale=S[side])
        for name, t, w, per in (("codes", cache.tensors[3 * side], want["codes"], D // 2),
                                ("scales", cache.tensors[3 * side + 1], want["scales"], D // block)):
            full = np.full((pages, H, page, per), 0xA5, np.uint8)
            full[at // page, :, at % page] = w.reshape(T, H, per)[kept]
            got = t.cpu().numpy()
            assert np.array_equal(got, full), f"{name} of side {side}: {np.sum(got != full)} bytes differ"
    # and back
    y = {}
    for dtype, od in ((torch.float32, ref.F32), (torch.bfloat16, ref.BF16)):
        y[dtype] = B.kv_read(cache, given.cuda(), dtype=dtype)
        for side in range(2):
            rows = host(x[side].contiguous().reshape(T * H, D))
            q = ref.quantize(rows, fmt=rf, rule=RULES[rule][1], window=window, rotate=block if rotate else 0,
                             global_scale=S[side])
            w = ref.dequantize(q["codes"], q["scales"], S[side], T * H, D, fmt=rf,
                               unrotate=block if rotate else 0, out_dtype=od).reshape(T, H, D)
            w[~kept] = 0
            assert np.array_equal(host(y[dtype][side]), w), f"read of side {side} as {dtype}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("fmt,rule", [("nvfp4", "absmax"), ("nvfp4", "sweep"), ("nvfp4", "foursix"),
                                      ("mxfp4", "absmax"), ("mxfp4", "sweep")])
def test_write_and_read(fmt, rule, rotate, dtype):
    rng = np.random.default_rng(11)
    for T, H, D, page in ((1, 1, 64, 16), (37, 3, 128, 16), (130, 2, 256, 48), (5, 8, 64, 1)):
        x = [torch.from_numpy(values(rng, (T, H, D))) for _ in range(2)]
        x = [t.to(torch.bfloat16) if dtype == "bf16" else t for t in x]
        write_and_check(rng, x, fmt, rule, rotate, page=page)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_strides_and_dropped_slots(fmt):
    rng = np.random.default_rng(12)
    for dtype in (torch.float32, torch.bfloat16):
        x = [torch.from_numpy(values(rng, (29, 5, 128))).to(dtype) for _ in range(2)]
        write_and_check(rng, x, fmt, "absmax", strided=True, drop=[(0, -1), (7, 0), (28, 1 << 40), (13, -(1 << 62))])


def test_sweep_on_ties_zeros_and_ends_of_the_scale_range():
    """Blocks of grid values (many equal errors), zero blocks, single spikes, and blocks whose AbsMax pattern lies at
    either end of E4M3 under the given global scale."""
    rng = np.random.default_rng(13)
    T, H, D = 64, 2, 128
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
    x = grid[rng.integers(0, 8, (T, H, D))] * rng.choice([-1, 1], (T, H, D)).astype(np.float32)
    x *= np.exp2(rng.integers(-12, 6, (T, H, 1))).astype(np.float32)
    x[::7] = 0
    x[3::7, :, 1:] = 0
    x[5::7] *= 1e4
    for S in ((0.01, 1.0), (2.0 ** -20, 64.0)):
        t = [torch.from_numpy(x.astype(np.float32)), torch.from_numpy(x[::-1].copy())]
        write_and_check(rng, t, "nvfp4", "sweep", S=S)
        write_and_check(rng, [as_bf16(x), as_bf16(x[::-1].copy())], "nvfp4", "sweep", rotate=True, S=S)


@pytest.mark.parametrize("window", [(0, 0), (-126, 126), (2, 5), (-8, 7), (-20, -10)])
def test_sweep_windows(window):
    rng = np.random.default_rng(14)
    x = [torch.from_numpy(values(rng, (19, 2, 64))) for _ in range(2)]
    write_and_check(rng, x, "nvfp4", "sweep", window=window)
    if window[1] - window[0] < 30:
        write_and_check(rng, x, "mxfp4", "sweep", window=window)


def test_many_tokens_agree_with_the_quantizer():
    """A long prompt, swept and rotated: the bytes of fp4q_quantize of the same rows."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, D, page = 5000, 4, 128, 64
    x = [torch.randn(T, H, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    pages = -(-T // page)
    S = [float(t.float().abs().max()) * 1.3 / 1536 for t in x]
    cache = B.alloc_kv_cache(pages, H, page, D, *S, scale_rule=B.FP4Q_SCALE_SWEEP, rotate=16)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    B.kv_write(cache, x[0], x[1], slots)
    for side in range(2):
        codes, scales, _ = B.quantize(x[side].reshape(T * H, D), scale_rule=B.FP4Q_SCALE_SWEEP, rotate=16,
                                      global_scale=S[side])
        at, off = slots // page, slots % page
        assert torch.equal(cache.tensors[3 * side][at, :, off].reshape(-1), codes)
        assert torch.equal(cache.tensors[3 * side + 1][at, :, off].reshape(-1), scales)


def test_empty_calls_do_nothing():
    cache = B.alloc_kv_cache(2, 1, 16, 64, 1.0, 1.0)
    none = torch.empty(0, 1, 64, device="cuda")
    B.kv_write(cache, none, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    k, v = B.kv_read(cache, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)
