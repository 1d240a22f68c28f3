"""What the binding says of a product's workspace before the call (no GPU needed)."""
import os

import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

if not os.path.exists(B.LIB_PATH):
    pytest.skip("libfp4q.so not built", allow_module_level=True)


def weight(rows=40, cols=64, **kw):
    return B.QuantizedWeight(torch.zeros(rows * cols // 2, dtype=torch.uint8), torch.zeros(rows * cols // 16, dtype=torch.uint8),
                             torch.ones(1), rows, cols, require_cuda=False, **kw)


def test_types_that_no_call_takes():
    w = weight()
    assert B.matmul_workspace_bytes(w, 50, torch.float32) > B.matmul_workspace_bytes(w, 50) >= 0
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError):
            B.matmul_workspace_bytes(w, 50, dtype)
        with pytest.raises(ValueError):
            B.gated_workspace_bytes(w, w, 50, dtype)


def test_pairs_that_no_call_takes():
    for other in (weight(48), weight(40, 128), weight(rotate=16)):
        with pytest.raises(ValueError):
            B.gated_workspace_bytes(weight(), other, 50, torch.float32)
