"""Writing into the 4-bit KV cache at the ends of binary32: global scales at the ends of their range, values from
denormals to the largest, every rule, every byte against the CPU oracle."""
import numpy as np
import pytest
import torch

from test_gpu_kv_rows import write_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("rule", ["absmax", "sweep", "foursix"])
@pytest.mark.parametrize("S", [(2.0 ** -117, 2.0 ** 119), (2.0 ** -100, 2.0 ** 100), (2.0 ** -60, 2.0 ** 60)])
def test_global_scales_at_their_ends(S, rule, rotate):
    rng = np.random.default_rng(91)
    for dtype in (torch.float32, torch.bfloat16):
        x = []
        for s in S:
            t = rng.standard_normal((40, 2, 128)) * np.exp2(rng.uniform(-14, 11, (40, 2, 1))) * s
            x.append(torch.from_numpy(np.clip(t, -2.0 ** 122, 2.0 ** 122).astype(np.float32)).to(dtype))
        write_and_check(rng, x, "nvfp4", rule, rotate, S=S)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("rule,window", [("absmax", None), ("sweep", None), ("sweep", (-3, 3)), ("sweep", (-126, 126))])
def test_exponents_at_their_ends(rule, window, rotate):
    rng = np.random.default_rng(92)
    for dtype in (torch.float32, torch.bfloat16):
        x = []
        for at in (-149, 122):
            t = rng.standard_normal((24, 2, 64)) * np.exp2(at + rng.uniform(-2, 24, (24, 2, 1)) * (1 if at < 0 else -1))
            x.append(torch.from_numpy(np.clip(t, -2.0 ** 122, 2.0 ** 122).astype(np.float32)).to(dtype))
        write_and_check(rng, x, "mxfp4", rule, rotate, window=window)
