"""Attention under global scales at the ends of their documented range, [2^-117, 2^119]: the same relative bounds as at
ordinary scales."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu

# few queries in one workgroup and over several, many in one launch and joined
CALLS = [([1, 1], [150, 77]), ([1, 1], [5000, 300]), ([60, 40], [150, 77]), ([40, 33], [9001, 300])]


def times(f, side, up):
    """The global scale of a side, and its values, times 2^up."""
    f.S[side] = np.float32(f.S[side] * 2.0 ** up)
    assert 2.0 ** -117 <= f.S[side] <= 2.0 ** 119
    for kv in f.kv:
        kv[side] = kv[side] * 2.0 ** up


def run(f, q, q_lens, what, **kw):
    st = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    want = attention64(f, q.double().numpy(), st, bf16=q.dtype == torch.bfloat16, **kw)
    out, lse = B.attend(f.cache(), q.cuda(), torch.tensor(f.lens, dtype=torch.int32, device="cuda"),
                        block_table=f.device_table(), q_starts=torch.from_numpy(st).cuda(), max_q=max(q_lens),
                        return_lse=True, **kw)
    torch.cuda.synchronize()
    check(out, lse, *want, what=what)


def first_values_only(f, code, byte, dims=1):
    """K rows whose first `dims` elements are alike and the others zero: `code` (magnitudes of E2M1) and scale `byte` by
    key."""
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    for b, n in enumerate(f.lens):
        key = np.arange(n)
        page, at = f.table[b, key // f.page], key % f.page
        f.codes[0][page, :, at] = 0
        if dims == 1:
            f.codes[0][page, :, at, 0] = code[:n, None]
        else:
            f.codes[0][page, :, at, :dims // 2] = 17 * code[:n, None, None]
        f.scales[0][page, :, at] = byte[:n, None, None]
        scale = torch.from_numpy(byte[:n].copy()).view(torch.float8_e4m3fn).float().numpy()
        f.kv[b][0] = np.zeros_like(f.kv[b][0])
        f.kv[b][0][:, :, :dims] = (grid[code[:n]] * (scale * f.S[0]).astype(np.float64))[:, None]


@pytest.mark.parametrize("k_up,v_up,q_up", [(0, -110, 0), (0, 110, 0), (-110, 0, 112), (110, 0, -110), (-60, -60, 60)])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ends_of_the_scale_range(dtype, rotate, k_up, v_up, q_up):
    """Both scales times powers of two, queries the other way."""
    rng = np.random.default_rng(51)
    for q_lens, lens in CALLS:
        f = Filled(rng, "nvfp4", 64, 1, 64, lens, rotate)
        for s, up in enumerate((k_up, v_up)):
            times(f, s, up)
        q = torch.from_numpy((rng.standard_normal((sum(q_lens), 2, 64)) * 2.0 ** q_up).astype(np.float32))
        q = q.to(torch.bfloat16) if dtype == "bf16" else q
        run(f, q, q_lens, f"{q_lens} {lens}")


@pytest.mark.parametrize("q_lens,lens", [([1], [256]), ([1], [9216]), ([96], [500]), ([96], [9216])])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_values_under_large_sums(dtype, rotate, q_lens, lens):
    """V's scale at the low end, and logits that stay 5.9 (in log2 units) above the first ones of every 256 keys, so
    that the sum of probabilities reaches thousands of times the largest that a running maximum would leave."""
    rng = np.random.default_rng(54)
    f = Filled(rng, "nvfp4", 64, 1, 64, lens, rotate)
    times(f, 1, -111)
    key = np.arange(max(lens))
    first_values_only(f, np.where(key % 256 < 128, 0, 7).astype(np.uint8), np.full(len(key), 0x38, np.uint8))
    q = np.zeros((sum(q_lens), 1, 64), np.float32)
    q[:, :, :16 if rotate else 1] = (5.9 / 1.4427 / (6 * f.S[0] / 8)) / (4 if rotate else 1)  # rotated: element 0
    q = torch.from_numpy(q)
    run(f, q.to(torch.bfloat16) if dtype == "bf16" else q, q_lens, f"{q_lens} {lens}")


@pytest.mark.parametrize("q_lens,lens", [([1], [256]), ([96], [500])])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_keys_large_queries_small_scale(dtype, q_lens, lens):
    """K's scale at the low end, queries at the high end of binary32, and a scale of 99 * 2^-33: logits of about 1."""
    rng = np.random.default_rng(55)
    f = Filled(rng, "nvfp4", 64, 1, 64, lens)
    times(f, 0, -110)
    n = max(lens)
    first_values_only(f, rng.integers(1, 8, n).astype(np.uint8), rng.integers(0x60, 0x7F, n).astype(np.uint8), 64)
    q = 2.0 ** 126 * rng.uniform(0.5, 1.0, (sum(q_lens), 1, 64)) * rng.choice([-1, 1], (sum(q_lens), 1, 1))
    q = torch.from_numpy(q.astype(np.float32))
    run(f, q.to(torch.bfloat16) if dtype == "bf16" else q, q_lens, f"{q_lens} {lens}", scale=99 * 2.0 ** -33)
