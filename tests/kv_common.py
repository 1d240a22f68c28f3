"""What the KV-cache tests share: caches with known bytes, and attention in 64 bits (numpy, on the host) with bounds on
how far a result of the kernels' arithmetic may lie from it."""
import math

import numpy as np
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from oracle import ref

FMT = {"nvfp4": (B.FP4Q_NVFP4, ref.NVFP4, 16), "mxfp4": (B.FP4Q_MXFP4, ref.MXFP4, 32)}
U32, UF16, UBF16 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8  # half a step, relative


def values(rng, shape, spread=0.5):
    """Normal values with a scale of its own per row and a few large ones."""
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    x[rng.random(shape) < 0.002] *= 20
    return x.astype(np.float32)


def as_bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16)


class Filled:
    """A cache whose pages hold quantized rows; `rows(b, n)` gives a sequence's K and V in 64 bits, in the domain they
    are stored in.  layout: "hnd" [pages, heads, tokens], "nhd" [pages, tokens, heads] or "both" (K and V of a page in one
    allocation).  Rows that no sequence holds are filled with bytes of the worst kind (NaN scales)."""

    def __init__(self, rng, fmt, dim, heads, page, lens, rotate=False, contiguous=False, layout="hnd", spare=2):
        f, rf, block = FMT[fmt]
        self.fmt, self.dim, self.heads, self.page, self.block, self.lens = fmt, dim, heads, page, block, lens
        need = [1 if contiguous else -(-n // page) for n in lens]
        pages = max(1, sum(need) + (0 if contiguous else spare))
        order = np.arange(pages) if contiguous else rng.permutation(pages)
        self.table = None if contiguous else np.full((len(lens), max(need + [1])), -1, np.int32)
        codes = [rng.integers(0, 256, (pages, heads, page, dim // 2), dtype=np.uint8) for _ in range(2)]
        scales = [np.full((pages, heads, page, dim // block), 0xFF, np.uint8) for _ in range(2)]
        self.S = [np.float32(0.011), np.float32(0.017)]
        self.kv = []  # per sequence, per side: [heads, n, dim] in 64 bits
        at = 0
        for b, n in enumerate(lens):
            got = order[at:at + need[b]]
            at += need[b]
            if self.table is not None:
                self.table[b, :need[b]] = got
            sides = []
            for s in range(2):
                x = values(rng, (heads, n, dim))
                if n:
                    qz = ref.quantize(x.reshape(-1, dim), fmt=rf, global_scale=float(self.S[s]))
                    c = qz["codes"].reshape(heads, n, dim // 2)
                    sc = qz["scales"].reshape(heads, n, dim // block)
                    y = ref.dequantize(qz["codes"], qz["scales"], float(self.S[s]), heads * n, dim, fmt=rf)
                    for j in range(need[b]):
                        m = min(page, n - j * page)
                        codes[s][got[j], :, :m] = c[:, j * page:j * page + m]
                        scales[s][got[j], :, :m] = sc[:, j * page:j * page + m]
                else:
                    y = np.zeros((0, dim), np.float32)
                sides.append(y.reshape(heads, n, dim).astype(np.float64))
            self.kv.append(sides)
        self.codes, self.scales = codes, scales
        self.rotate = block if rotate else 0
        self.layout, self.format = layout, f

    def cache(self, device="cuda"):
        def put(pair):
            if self.layout == "nhd":
                return [torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3))).to(device).transpose(1, 2)
                        for x in pair]
            if self.layout == "both":
                both = torch.from_numpy(np.stack(pair, 1)).to(device)
                return [both[:, 0], both[:, 1]]
            return [torch.from_numpy(x).to(device) for x in pair]

        (kc, vc), (ks, vs) = put(self.codes), put(self.scales)
        g = [torch.tensor([s], dtype=torch.float32, device=device) if self.fmt == "nvfp4" else None for s in self.S]
        return B.KvCache(kc, ks, g[0], vc, vs, g[1], format=self.format, rotate=self.rotate,
                         require_cuda=device == "cuda")

    def device_table(self, device="cuda"):
        return None if self.table is None else torch.from_numpy(self.table).to(device)


def sylvester(n):
    h = np.ones((1, 1))
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(n)


def blocks_times(x, n):
    return (x.reshape(-1, n) @ sylvester(n)).reshape(x.shape)


def attention64(f, q, q_starts, causal=True, window=0, scale=None, bf16=True):
    """(out, lse, bound of |error| of out, bound of |error| of lse) of the queries q [total, Hq, D] (64 bits), and which
    rows belong to a sequence.

    The bounds follow the arithmetic.  A logit x = scale sum_d q_d k_d is summed in binary32 over D products (and over
    the parts of q, whose remainder is below 2^-21 of an element): off by at most
    (D + 8) u32 + 2^-21 times scale sum |q_d k_d|, and by a few u32 |x| from its factor and exponent.  A probability is
    then off by twice that, relatively, plus a few u32, plus the rounding of its parts: half a step of f16 (NVFP4) or the
    square of bf16's (two parts, MXFP4) for bf16 results, the square or the cube for binary32 results, never less than
    u32; sums over n keys add (n + 16) u32.  All of it is relative to A = sum p |v|.  What is below 2^-33 of the largest
    probability may be lost: n 2^-32 max|v|.  The rotation of the result adds (block + 2) u32 of sum |o|.  The result's
    own rounding adds half a step of its type."""
    total, Hq, D = q.shape
    G = Hq // f.heads
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((total, Hq, D)), np.full((total, Hq), -np.inf)
    tol, ltol = np.zeros((total, Hq, D)), np.zeros((total, Hq))
    own = np.zeros(total, bool)
    part = {("nvfp4", True): UF16, ("mxfp4", True): UBF16 ** 2, ("nvfp4", False): UF16 ** 2,
            ("mxfp4", False): UBF16 ** 3}[f.fmt, bf16] + 2 * U32
    for b, m in enumerate(f.lens):
        r0, r1 = int(q_starts[b]), int(q_starts[b + 1])
        n = r1 - r0
        own[r0:r1] = True
        pos = np.arange(n)[:, None] + (m - n)
        key = np.arange(m)[None]
        seen = (key <= pos) if causal else np.ones((n, m), bool)
        if window:
            seen &= key > pos - window
        for h in range(Hq):
            k, v = f.kv[b][0][h // G], f.kv[b][1][h // G]
            x = q[r0:r1, h]
            if f.rotate:
                x = blocks_times(x, f.rotate)
            w = np.where(seen, scale * (x @ k.T), -np.inf)
            mass = np.where(seen, abs(scale) * (np.abs(x) @ np.abs(k).T), 0)
            top = w.max(-1, initial=-np.inf, keepdims=True)
            some = np.isfinite(top)
            p = np.where(seen, np.exp(w - np.where(some, top, 0)), 0)
            l = p.sum(-1, keepdims=True)
            pn = p / np.where(l > 0, l, 1)
            o = pn @ v
            A = pn @ np.abs(v)
            off = ((D + 8) * U32 + 2.0 ** -21) * mass.max(-1, initial=0) + \
                8 * U32 * np.abs(np.where(seen, w, 0)).max(-1, initial=0) + 8 * U32
            rel = 2 * off + part + (m + 16) * U32
            lost = m * 2.0 ** -32 * np.abs(v).max(initial=0)
            t = rel[:, None] * A + lost
            if f.rotate:
                o = blocks_times(o, f.rotate)
                c = f.rotate ** -0.5
                t = np.repeat(c * t.reshape(n, -1, f.rotate).sum(-1), f.rotate, -1).reshape(n, D) + \
                    np.repeat(c * (f.rotate + 2) * U32 * np.abs(A).reshape(n, -1, f.rotate).sum(-1), f.rotate,
                              -1).reshape(n, D)
            step = (UBF16 if bf16 else U32)
            out[r0:r1, h] = o
            tol[r0:r1, h] = t + step * (np.abs(o) + t) + (2.0 ** -133 if bf16 else 2.0 ** -149)
            with np.errstate(divide="ignore"):
                ls = (np.where(some, top, 0) + np.log(l))[:, 0]
            lse[r0:r1, h] = ls
            ltol[r0:r1, h] = off + (m + 16) * U32 + 8 * U32 * np.abs(np.where(np.isfinite(ls), ls, 0))
    return out, lse, tol, ltol, own


def check(got, lse, want, wlse, tol, ltol, own, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got[own])), f"{what}: not finite"
    over = np.abs(got - want)[own] - tol[own]
    assert over.max(initial=-1) <= 0, f"{what}: out is {over.max():.3g} over its bound (of {tol[own].max():.3g})"
    empty = ~np.isfinite(wlse) & own[:, None]
    assert np.all(np.isneginf(lse[empty])), f"{what}: lse of empty rows"
    assert np.all(got[empty] == 0), f"{what}: out of empty rows"
    full = np.isfinite(wlse) & own[:, None]
    over = np.abs(lse[full] - wlse[full]) - ltol[full]
    assert over.max(initial=-1) <= 0, f"{what}: lse is {over.max():.3g} over its bound"
