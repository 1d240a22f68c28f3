"""Attention under bounds far above the lengths there are."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_kv", [131072, 1 << 22])
def test_many_pairs_under_a_long_bound(max_kv):
    """512 sequences of 32 heads, short but for one: the bound asks for more steps than a launch has workgroups, the
    lengths for few."""
    rng = np.random.default_rng(81)
    lens = [int(n) for n in rng.integers(0, 20, 512)]
    lens[300] = 700
    f = Filled(rng, "nvfp4", 64, 32, 16, lens)
    q = torch.from_numpy(rng.standard_normal((512, 32, 64)).astype(np.float32)).to(torch.bfloat16)
    want = attention64(f, q.double().numpy(), np.arange(513))
    out, lse = B.attend(f.cache(), q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max_kv=max_kv,
                        block_table=f.device_table(), return_lse=True)
    check(out, lse, *want, what=str(max_kv))


@pytest.mark.parametrize("batch", [3, 300])
def test_a_loose_bound_of_queries(batch):
    """Packed prompts without max_q: the rows of all sequences are each one's bound."""
    rng = np.random.default_rng(82)
    q_lens = [int(n) for n in rng.integers(0, 5, batch)]
    q_lens[1] = 90
    lens = [n + int(rng.integers(0, 40)) for n in q_lens]
    f = Filled(rng, "mxfp4", 64, 2, 16, lens)
    st = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((st[-1], 4, 64)).astype(np.float32)).to(torch.bfloat16)
    out, lse = B.attend(f.cache(), q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                        block_table=f.device_table(), q_starts=torch.from_numpy(st).cuda(), return_lse=True)
    check(out, lse, *attention64(f, q.double().numpy(), st), what=str(batch))
