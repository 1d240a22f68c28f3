"""New tokens' rows as the definition of the cache's append gives them, in numpy binary32 (and binary64 for the norm), and the
bytes that the oracle makes of them."""
import numpy as np
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from oracle import ref

FMT = {"nvfp4": (B.FP4Q_NVFP4, ref.NVFP4, 16), "mxfp4": (B.FP4Q_MXFP4, ref.MXFP4, 32)}
RULE = {"absmax": (B.FP4Q_SCALE_ABSMAX, ref.ABSMAX), "sweep": (B.FP4Q_SCALE_SWEEP, ref.SWEEP),
        "foursix": (B.FP4Q_SCALE_FOUR_OVER_SIX, ref.FOUR_SIX)}


def turned(x, weight, eps, table, positions, interleaved):
    """Rows x [tokens, heads, dim] (binary32 numpy), normed and turned: each product and sum rounded to binary32."""
    x = x.astype(np.float32)
    if weight is not None:
        mean = np.square(x.astype(np.float64)).sum(-1) / x.shape[-1]
        r = (1.0 / np.sqrt(mean + np.float64(np.float32(eps)))).astype(np.float32)
        x = (x * r[..., None]) * weight.astype(np.float32)
    if table is None:
        return x
    R = table.shape[1]
    good = (positions >= 0) & (positions < table.shape[0])
    row = table[np.where(good, positions, 0)][:, None] if table.shape[0] else np.zeros((len(positions), 1, R), np.float32)
    c, s = row[..., :R // 2], row[..., R // 2:]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    p, q = a * c - b * s, b * c + a * s
    out = x.copy()
    if interleaved:
        out[..., 0:R:2], out[..., 1:R:2] = p, q
    else:
        out[..., :R // 2], out[..., R // 2:R] = p, q
    out[~good] = np.nan
    return out


def as_type(x, dtype):
    """Binary32 rows rounded to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)


def bytes_of(x, fmt, rule, S, rotate, window=None):
    """(codes, scales) of rows [..., dim] by the oracle."""
    f, rf, block = FMT[fmt]
    kw = {} if window is None else dict(window=window)
    q = ref.quantize(np.ascontiguousarray(x.reshape(-1, x.shape[-1])), fmt=rf, rule=RULE[rule][1], rotate=block if rotate else 0,
                     global_scale=float(S), **kw)
    return q["codes"].reshape(*x.shape[:-1], -1), q["scales"].reshape(*x.shape[:-1], -1)
