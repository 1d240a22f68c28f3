"""Attention with a window over caches whose rows before the window hold bytes of the worst kind: no query sees them, so
nothing of them may show, wherever the window starts within a page or a tile."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu


def spoil(f, first, byte):
    """Rows below key first[b] of sequence b get `byte` as every scale and 0xFF codes; pages wholly below it become other
    (valid) pages that hold nothing but NaN."""
    used = set() if f.table is None else set(f.table[f.table >= 0].tolist())
    spare = [p for p in range(len(f.codes[0])) if p not in used]
    for b, n in enumerate(first):
        for s in range(2):
            for j in range(0, n, f.page):
                page = b if f.table is None else f.table[b, j // f.page]
                f.scales[s][page, :, :min(f.page, n - j)] = byte
                f.codes[s][page, :, :min(f.page, n - j)] = 0xFF
        if f.table is not None:
            f.table[b, :n // f.page] = spare[0]


@pytest.mark.parametrize("byte", [0xFF, "other"])
@pytest.mark.parametrize("contiguous", [False, True])
@pytest.mark.parametrize("q_len", [1, 4, 90, 300])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_before_the_window(fmt, q_len, contiguous, byte):
    """Starts of the window at 0, 1, 15, 16, 17 and 31 past a tile of 32 keys, and behind several of them."""
    rng = np.random.default_rng(41)
    byte = {"nvfp4": 0x7F, "mxfp4": 0xFE}[fmt] if byte == "other" else byte  # the other NaN; 6 * 2^127
    first = [0, 1, 15, 16, 17, 31, 32 + 15, 320 + 17, 2048 + 31]
    window = 45
    lens = [n + window + q_len - 1 for n in first]
    for dim, page, group in ((64, 16, 2), (128, 48, 2), (256, 16, 1)):
        if contiguous:
            page = max(lens)
        f = Filled(rng, fmt, dim, 2, page, lens, contiguous=contiguous)
        total = q_len * len(lens)
        q = torch.from_numpy(rng.standard_normal((total, 2 * group, dim)).astype(np.float32)).to(torch.bfloat16)
        want = attention64(f, q.double().numpy(), np.arange(len(lens) + 1) * q_len, window=window)
        spoil(f, first, byte)
        out, lse = B.attend(f.cache(), q.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                            block_table=f.device_table(), window=window, return_lse=True)
        check(out, lse, *want, what=f"{fmt} {dim} {q_len}")
