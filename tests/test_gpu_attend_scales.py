"""Attention under global scales that are not finite, and under negative ones."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu

# few queries in one workgroup and over several, many in one launch and joined
CALLS = [([1, 1], [150, 77]), ([1, 1], [5000, 300]), ([60, 40], [150, 77]), ([40, 33], [9001, 300])]


def attend(f, q, q_lens, **kw):
    st = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    out, lse = B.attend(kw.pop("cache", None) or f.cache(), q.cuda(),
                        torch.tensor(f.lens, dtype=torch.int32, device="cuda"), block_table=f.device_table(),
                        q_starts=torch.from_numpy(st).cuda(), max_q=max(q_lens), return_lse=True, **kw)
    torch.cuda.synchronize()
    return st, out, lse


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_scale_that_is_not_finite_shows(side, bad):
    """NaN in every row that sees a key, zeros in those that do not."""
    rng = np.random.default_rng(52)
    for q_lens, lens in CALLS + [([3, 2], [1, 40]), ([70, 9], [20, 40])]:
        f = Filled(rng, "nvfp4", 64, 1, 64, lens)
        f.S[side] = np.float32(bad)
        q = torch.from_numpy(rng.standard_normal((sum(q_lens), 2, 64)).astype(np.float32)).to(torch.bfloat16)
        st, out, lse = attend(f, q, q_lens)
        for b, n in enumerate(lens):
            none = max(0, q_lens[b] - n)
            o, l = out[st[b]:st[b + 1]], lse[st[b]:st[b + 1]]
            assert torch.all(o[:none] == 0) and torch.all(torch.isneginf(l[:none]))
            assert not torch.any(torch.isfinite(o[none:]).all(-1)), (q_lens, lens, b)
            if side == 0:
                assert torch.all(torch.isnan(o[none:])) and torch.all(torch.isnan(l[none:]))


def test_negative_scales():
    """A negative global scale is the sign of every value."""
    rng = np.random.default_rng(53)
    for q_lens, lens in CALLS:
        f = Filled(rng, "nvfp4", 64, 1, 64, lens)
        for s in range(2):
            f.S[s] = np.float32(-f.S[s])
            for kv in f.kv:
                kv[s] = -kv[s]
        q = torch.from_numpy(rng.standard_normal((sum(q_lens), 2, 64)).astype(np.float32))
        for scale in (None, -0.2):
            st, out, lse = attend(f, q, q_lens, scale=scale)
            check(out, lse, *attention64(f, q.double().numpy(), st, scale=scale, bf16=False))
