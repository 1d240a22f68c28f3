"""Attention over MXFP4 caches whose exponents reach the low end of E8M0, and far up: the same relative bounds as at
ordinary ones."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu


def shift(f, side, up):
    """A side's values times 2^up; up None: so far down that the least exponent byte becomes 0."""
    live = [(b, j) for b, n in enumerate(f.lens) for j in range(-(-n // f.page))]
    places = [(f.table[b, j], min(f.page, f.lens[b] - j * f.page)) for b, j in live]
    if up is None:
        up = -int(min(f.scales[side][p, :, :m].min() for p, m in places))
    for p, m in places:
        by = f.scales[side][p, :, :m].astype(int) + up
        assert by.min() >= 0 and by.max() < 255
        f.scales[side][p, :, :m] = by
    for kv in f.kv:
        kv[side] = kv[side] * 2.0 ** up
    return up


@pytest.mark.parametrize("k_up,v_up", [(0, None), (None, 0), (0, 90), (90, 0), (-60, 60)])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ends_of_the_exponents(dtype, rotate, k_up, v_up):
    rng = np.random.default_rng(71)
    for q_lens, lens in (([1, 1], [150, 77]), ([1, 1], [5000, 300]), ([60, 40], [150, 77]), ([40, 33], [9001, 300])):
        f = Filled(rng, "mxfp4", 64, 1, 64, lens, rotate)
        up = shift(f, 0, k_up)
        shift(f, 1, v_up)
        # the transform sums a block of queries before its factor: they stay below 2^127 / 32
        q = torch.from_numpy((rng.standard_normal((sum(q_lens), 2, 64)) * 2.0 ** min(-up, 115)).astype(np.float32))
        q = q.to(torch.bfloat16) if dtype == "bf16" else q
        st = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        want = attention64(f, q.double().numpy(), st, bf16=dtype == "bf16")
        out, lse = B.attend(f.cache(), q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                            block_table=f.device_table(), q_starts=torch.from_numpy(st).cuda(), max_q=max(q_lens),
                            return_lse=True)
        check(out, lse, *want, what=f"{q_lens} {lens}")
