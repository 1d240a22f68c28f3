"""Prompts whose keys are cut into so many chunks that several groups of lanes join one row's partial results."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dim,keys", [(64, 20000), (128, 16401), (256, 9011)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_of_many_chunks(fmt, dim, keys, rotate, dtype):
    rng = np.random.default_rng(61)
    q_lens, lens = [96, 70], [keys, 77]
    f = Filled(rng, fmt, dim, 1, 64, lens, rotate)
    q = torch.from_numpy(rng.standard_normal((sum(q_lens), 1, dim)).astype(np.float32))
    q = q.to(torch.bfloat16) if dtype == "bf16" else q
    st = np.array([0, 96, 166], np.int32)
    args = dict(block_table=f.device_table(), q_starts=torch.from_numpy(st).cuda(), max_q=96)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = f.cache()
    need = B.attend_workspace_bytes(cache, q.cuda(), kv, **args)
    chunks = need // (len(lens) * 96 * (dim * 4 + 8))  # partial results of each row
    assert chunks > 4 * (256 // (dim // 4)), "the cut that this test is for"
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # places that hold nothing are NaN
    out, lse = B.attend(cache, q.cuda(), kv, return_lse=True, workspace=ws, **args)
    check(out, lse, *attention64(f, q.double().numpy(), st, bf16=dtype == "bf16"), what=f"{fmt} {dim} {chunks}")
