"""The 4-bit KV cache's operators, as measured: writing tokens into the cache and reading rows back, and attention over
the cache for single tokens (or a few) and for whole prompts.

Each case is plain numbers; `prepare` makes the inputs on the GPU from a seed, `run` is one pass, in plain torch
operations or (`own`) through this package's entry points, `exact` the same from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SWEEP = (-3, 7)  # window of E4M3 patterns around the AbsMax one


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    def case(name, op, **kw):
        c = dict(name=name, op=op, fmt="nvfp4", rotate=False, dtype="bf16", heads=8, group=4, dim=128, page=64)
        c.update(kw)
        return c

    def cache(name, op, tokens, **kw):
        return case(name, op, **{**dict(tokens=tokens, rule="absmax", pages_free=0.25), **kw})

    def attend(name, batch, q_len, ctx, **kw):
        return case(name, "attend", **{**dict(batch=batch, q_len=q_len, ctx=ctx, spread=0.0, window=0), **kw})

    return [
        # one decode step's new token of each of 64 sequences, ScaleSweep with the rotation
        cache("write_step", "write", 64, rule="sweep", rotate=True, page=16),
        # a long prompt written at once, the same rule
        cache("write_prompt", "write", 8192, rule="sweep", rotate=True),
        # an odd number of binary32 tokens, MXFP4, small heads
        cache("write_odd_mx", "write", 1003, fmt="mxfp4", dtype="f32", dim=64, page=48),
        # a short prefix taken out of the cache (to hand it to another worker)
        cache("read_short", "read", 257, page=16),
        # every row of a long context taken out, un-rotated
        cache("read_long", "read", 65536, rotate=True),
        # one sequence, short context: the latency of a call
        attend("decode_one", 1, 1, 131, page=16),
        # an ordinary serving batch, contexts of different lengths, rotated
        attend("decode_batch", 32, 1, 8192, spread=0.9, rotate=True),
        # the KV-cache workload [64, 32, 4096, 128], contiguous, rotated: every head its own keys
        attend("decode_kv", 64, 1, 4096, heads=32, group=1, page=0, rotate=True),
        # a few drafted tokens checked at once over very long contexts
        attend("decode_draft_mx", 3, 4, 65521, fmt="mxfp4", heads=4, group=8, page=16, spread=0.4),
        # odd short prompts packed together, binary32, small heads
        attend("prompt_odd_f32", 5, 213, 213, dtype="f32", dim=64, page=32, spread=0.95),
        # one chunk of a prompt after a long cached prefix
        attend("prompt_chunk_mx", 2, 509, 16384, fmt="mxfp4", spread=0.2),
        # a whole long prompt
        attend("prompt_long", 1, 8192, 8192, heads=8, group=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    c = dict(op=op, fmt=rng.choice(["nvfp4", "nvfp4", "mxfp4"]), rotate=rng.random() < 0.5,
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), heads=rng.choice([1, 2, 3, 4, 8, 16, 32]),
             group=rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]), dim=rng.choice([64, 128, 128, 128, 256]),
             page=rng.choice([0, 16, 32, 48, 64, 128, 256]))
    if op != "attend":
        most = (1 << 26) // (c["heads"] * c["dim"])
        c.update(page=c["page"] or 16, tokens=_log(rng, 1, min(65536, most)), pages_free=rng.uniform(0.0, 0.5),
                 rule=rng.choice(["absmax", "sweep"]) if c["fmt"] == "nvfp4" else "absmax")
        if c["rule"] == "sweep":
            c["tokens"] = min(c["tokens"], (1 << 23) // (c["heads"] * c["dim"]))
        return c
    spread = rng.choice([0.0, 0.5, 0.95]) * rng.uniform(0.5, 1.0)
    if rng.random() < 0.5:  # a few queries for each sequence
        batch, q_len = _log(rng, 1, 128), rng.choice([1, 1, 1, 1, 2, 3, 4, 6])
        ctx = max(q_len, _log(rng, 1, 1 << 17))
    else:  # prompts, or chunks of them after a prefix
        batch, q_len = _log(rng, 1, 16), _log(rng, 8, 8192)
        ctx = q_len + (rng.choice([0, 1]) and _log(rng, 1, 32768))
    # not more than the largest listed ones: cache values, scores held by the plain form, and operations
    live = (64 * 32 * 4096 * 128) // (batch * c["heads"] * c["dim"])
    scores = (32 * 8192 * 4096) // (batch * q_len * c["heads"] * c["group"])
    work = (32 * 8192 * 4096 * 128) // (batch * q_len * c["heads"] * c["group"] * c["dim"])
    while min(live, scores, work) < 1 or q_len > min(live, scores, work):
        batch, q_len = max(1, batch // 2), max(1, q_len // 2)
        live = (64 * 32 * 4096 * 128) // (batch * c["heads"] * c["dim"])
        scores = (32 * 8192 * 4096) // (batch * q_len * c["heads"] * c["group"])
        work = (32 * 8192 * 4096 * 128) // (batch * q_len * c["heads"] * c["group"] * c["dim"])
    ctx = max(q_len, min(ctx, live, scores, work))
    c.update(batch=batch, q_len=q_len, ctx=ctx, spread=spread,
             window=_log(rng, 1, 4096) if rng.random() < 0.2 else 0)
    return c


def _block(c):
    return 32 if c["fmt"] == "mxfp4" else 16


def _lens(c):
    """(queries, keys) of each sequence: the first has the full lengths, the others less, up to `spread` of them."""
    part = [math.modf(b * 0.6180339887498949)[0] * c["spread"] for b in range(c["batch"])]
    q = [c["q_len"]] * c["batch"] if c["q_len"] <= 8 else [max(1, round(c["q_len"] * (1 - f))) for f in part]
    part = part[:1] + part[:0:-1]
    return q, [n + round((c["ctx"] - c["q_len"]) * (1 - f)) for n, f in zip(q, part)]


def _pairs(c):
    """Visible (query, key) pairs over all sequences, and the keys that some query sees."""
    pairs = keys = 0
    for n, m in zip(*_lens(c)):
        w = c["window"] or m
        first = m - n  # keys before the first query
        full = max(0, min(n, w - first - 1))  # queries that see every key up to their own
        pairs += full * (first + 1) + full * (full - 1) // 2 + (n - full) * w
        keys += min(m, w + n - 1)
    return pairs, keys


def work(c):
    size = 2 if c["dtype"] == "bf16" else 4
    row = c["heads"] * c["dim"]
    held = 0.5 + 1.0 / _block(c)  # bytes of the cache for each value
    if c["op"] != "attend":
        n = 2.0 * c["tokens"] * row
        reads = n * size if c["op"] == "write" else 0.0
        return {"bytes": reads + n * held + n * size + 8 * c["tokens"], "flops": n * 4}
    pairs, keys = _pairs(c)
    rows = sum(_lens(c)[0]) * c["heads"] * c["group"]
    return {"bytes": 2.0 * keys * row * held + rows * (2 * c["dim"] * size + 4),
            "flops": 4.0 * c["dim"] * pairs * c["heads"] * c["group"]}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _random(g, shape, head_axis):
    """Values like a KV cache's: normal, a scale of its own for each head, one in a thousand thirty times as large."""
    x = torch.randn(shape, generator=g, device=DEV)
    side = [1] * len(shape)
    side[head_axis] = shape[head_axis]
    x *= torch.exp(0.5 * torch.randn(side, generator=g, device=DEV))
    x[torch.rand(shape, generator=g, device=DEV) < 0.001] *= 30.0
    return x


def _butterflies(x, n):
    """The orthonormal Hadamard transform of each n values of the last axis, in binary32 butterflies of widths 1, 2, ..."""
    y, h = x.reshape(-1, n), 1
    while h < n:
        y = y.reshape(-1, n // (2 * h), 2, h)
        y = torch.cat((y[:, :, :1] + y[:, :, 1:], y[:, :, :1] - y[:, :, 1:]), 2).reshape(-1, n)
        h *= 2
    return (y * torch.tensor(n ** -0.5, dtype=torch.float32, device=x.device)).reshape(x.shape)


def _e2m1_code(y):
    """The code of the nearest E2M1 magnitude to y >= 0, ties to the even code."""
    return ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))


def _step(scales, S, fmt):
    """The binary32 step of each scale byte."""
    if fmt == "mxfp4":
        return torch.exp2(scales.double() - 127).float()
    return scales.view(torch.float8_e4m3fn).float() * S


def _quantize(x, S, fmt, rule):
    """(codes, scale bytes) of binary32 x, blocks along the last axis: the steps of the method, in binary32."""
    n = 32 if fmt == "mxfp4" else 16
    b = x.reshape(-1, n)
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
        scale, r = (e + 127).to(torch.uint8), torch.exp2(-e.double()).float()
    else:
        scale = (top.double() / (6.0 * S).double()).float().clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = scale.clamp(min=1)
        if rule == "sweep":  # every pattern of the window: the one of least binary64 error, the smaller on a tie
            window = torch.arange(SWEEP[0], SWEEP[1] + 1, device=x.device)
            tried = (scale.int() + window).clamp(1, 126).to(torch.uint8)
            D = _step(tried, S, fmt).unsqueeze(-1)
            q = _lut(x.device)[_e2m1_code(b.abs().unsqueeze(1) * (1.0 / D.double()).float()).int()] * D
            err = (b.abs().unsqueeze(1).double() - q.double()).square().sum(-1)
            tried = torch.where(err == err.amin(-1, keepdim=True), tried.int(), 255)
            scale = tried.amin(-1, keepdim=True).to(torch.uint8)
        r = (1.0 / _step(scale, S, fmt).double()).float()
        r = torch.where(top > 0, r, torch.ones_like(r))
        scale = torch.where(top > 0, scale, torch.zeros_like(scale))
    nib = _e2m1_code(b.abs() * r) | (torch.signbit(b).to(torch.uint8) << 3)
    nib = nib.reshape(*x.shape[:-1], -1, 2)
    return nib[..., 0] | (nib[..., 1] << 4), scale.reshape(*x.shape[:-1], -1)


def _lut(device):
    return torch.tensor(E2M1, device=device)


def _dequantize(codes, scales, S, fmt, rotated):
    """Binary32 values of code and scale bytes, un-rotated."""
    n = 32 if fmt == "mxfp4" else 16
    one = torch.cat((_lut(codes.device), -_lut(codes.device)))
    byte = torch.arange(256, device=codes.device)
    two = torch.stack((one[byte & 15], one[byte >> 4]), -1)
    x = two[codes.int()].reshape(*scales.shape, n) * _step(scales, S, fmt).unsqueeze(-1)
    x = x.reshape(*codes.shape[:-1], -1)
    return _butterflies(x, n) if rotated else x


def _fill(c, g, pages, page):
    """A cache of `pages` pages, filled: (codes, scales, S), in pieces where it is large."""
    n = _block(c)
    codes = torch.empty(pages, c["heads"], page, c["dim"] // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, c["heads"], page, c["dim"] // n, dtype=torch.uint8, device=DEV)
    S = None
    step = max(1, (1 << 25) // (c["heads"] * page * c["dim"]))
    head = torch.exp(0.5 * torch.randn(1, c["heads"], 1, 1, generator=g, device=DEV))
    for p in range(0, pages, step):
        x = _random(g, (min(step, pages - p), c["heads"], page, c["dim"]), 0) * head
        if c["rotate"]:
            x = _butterflies(x, n)
        S = (x.abs().max() / 1536).reshape(1) if S is None else S
        codes[p:p + step], scales[p:p + step] = _quantize(x, S, c["fmt"], "absmax")
    return codes, scales, S


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s = {"case": c, "dtype": dtype}
    if c["op"] != "attend":
        T, page = c["tokens"], c["page"]
        pages = -(-int(T * (1 + c["pages_free"])) // page) + 1
        s["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:T]
        if c["op"] == "read":
            s["k"], s["v"] = _fill(c, g, pages, page), _fill(c, g, pages, page)
            return s
        n = _block(c)
        for name in ("k", "v"):
            x = _random(g, (T, c["heads"], c["dim"]), 1).to(dtype)
            top = (_butterflies(x.float(), n) if c["rotate"] else x.float()).abs().max()
            s[name + "_new"] = x
            s[name] = (torch.zeros(pages, c["heads"], page, c["dim"] // 2, dtype=torch.uint8, device=DEV),
                       torch.zeros(pages, c["heads"], page, c["dim"] // n, dtype=torch.uint8, device=DEV),
                       (top / 1536).reshape(1))
        return s
    q, kv = _lens(c)
    s["q"] = torch.randn(sum(q), c["heads"] * c["group"], c["dim"], generator=g, device=DEV).to(dtype)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    starts = [0]
    for n in q:
        starts.append(starts[-1] + n)
    s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["max_q"], s["max_kv"] = max(q), max(kv)
    if c["page"] == 0:  # one page of the full length for each sequence
        s["table"], pages, page = None, c["batch"], c["ctx"]
    else:
        page = c["page"]
        need = [-(-n // page) for n in kv]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((c["batch"], max(need)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            s["table"][b, :n] = order[at:at + n]
            at += n
    s["k"], s["v"] = _fill(c, g, pages, page), _fill(c, g, pages, page)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def _cache(s):
    """The handle of the cache that a program keeps."""
    if "cache" not in s:
        from block_scaled_fp4_fp4q_amd import binding as B
        c = s["case"]
        s["cache"] = B.KvCache(
            *s["k"], *s["v"], format=B.FP4Q_MXFP4 if c["fmt"] == "mxfp4" else B.FP4Q_NVFP4,
            scale_rule=B.FP4Q_SCALE_SWEEP if c.get("rule") == "sweep" else B.FP4Q_SCALE_ABSMAX,
            rotate=_block(c) if c["rotate"] else 0)
    return s["cache"]


def run(s):
    c = s["case"]
    if own:
        from block_scaled_fp4_fp4q_amd import binding as B
        cache = _cache(s)
        if c["op"] != "attend":
            if c["op"] == "write":
                B.kv_write(cache, s["k_new"], s["v_new"], s["slots"])
            k, v = B.kv_read(cache, s["slots"], dtype=s["dtype"])  # what the cache now stands for
            return {"k": k, "v": v}
        out, lse = B.attend(cache, s["q"], s["kv_lens"], max_kv=s["max_kv"], block_table=s["table"],
                            q_starts=None if c["q_len"] <= 8 else s["q_starts"], max_q=s["max_q"], causal=True,
                            window=c["window"], return_lse=True)
        return {"out": out, "lse": lse}
    if c["op"] != "attend":
        return _plain_rows(s)
    return _plain_attend(s)


def _plain_rows(s):
    c, got = s["case"], {}
    n, page = _block(c), c["page"]
    at, off = s["slots"] // page, s["slots"] % page
    for name in ("k", "v"):
        codes, scales, S = s[name]
        if c["op"] == "write":
            x = s[name + "_new"].float()
            x = _butterflies(x, n) if c["rotate"] else x
            codes[at, :, off], scales[at, :, off] = _quantize(x, S, c["fmt"], c["rule"])
        x = _dequantize(codes[at, :, off], scales[at, :, off], S, c["fmt"], c["rotate"])
        got[name] = x.to(s["dtype"])
    return got


def _rows_of(s, name):
    """Binary32 values of every key or value of every sequence: [batch, heads, max_kv, dim]."""
    c = s["case"]
    codes, scales, S = s[name]
    if s["table"] is None:
        codes, scales = codes[:, :, :s["max_kv"]], scales[:, :, :s["max_kv"]]
    else:
        t = torch.arange(s["max_kv"], device=codes.device)
        at, off = s["table"].clamp(min=0)[:, t // c["page"]], t % c["page"]
        codes, scales = codes[at, :, off].transpose(1, 2), scales[at, :, off].transpose(1, 2)
    return _dequantize(codes.contiguous(), scales.contiguous(), S, c["fmt"], c["rotate"])


def _plain_attend(s):
    c, q = s["case"], s["q"]
    H, G, D, B = c["heads"], c["group"], c["dim"], c["batch"]
    Lq, Lk = s["max_q"], s["max_kv"]
    row = torch.arange(q.shape[0], device=q.device)
    starts = s["q_starts"].long()
    b = torch.bucketize(row, starts[1:], right=True)
    i = row - starts[b]
    pad = torch.zeros(B, Lq, H, G, D, device=q.device)
    pad[b, i] = q.float().reshape(-1, H, G, D)
    pad = pad.permute(0, 2, 3, 1, 4).reshape(B, H, G * Lq, D)
    w = torch.matmul(pad, _rows_of(s, "k").transpose(2, 3).contiguous()).reshape(B, H, G, Lq, Lk)
    w *= D ** -0.5
    where = (s["kv_lens"] - (starts[1:] - starts[:-1]))[:, None, None] + torch.arange(Lq, device=q.device)[:, None]
    key = torch.arange(Lk, device=q.device)
    seen = (key <= where) & (key < s["kv_lens"][:, None, None])
    if c["window"]:
        seen &= key > where - c["window"]
    w.masked_fill_(~seen[:, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(m.clamp(min=-3e38)).exp_()
    l = w.sum(-1, keepdim=True)
    out = torch.matmul(w.reshape(B, H, G * Lq, Lk), _rows_of(s, "v")).reshape(B, H, G, Lq, D)
    out = torch.where(l > 0, out / l, torch.zeros_like(out))
    lse = (m + torch.log(l)).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4)[b, i].reshape(q.shape)
    return {"out": out.to(s["dtype"]), "lse": lse.permute(0, 3, 1, 2)[b, i].reshape(q.shape[0], H * G)}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _sylvester(n):
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while h.shape[0] < n:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(n)


def _exact_values(codes, scales, S, c):
    """Values of cache rows in 64 bits: sign, magnitude, the step fl32(s S) or 2^e, and the rotation undone."""
    n = _block(c)
    nib = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).long()
    e, f = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.exp2((e - 1).double()))
    x = torch.where(nib >= 8, -mag, mag)
    by = scales.long()
    if c["fmt"] == "mxfp4":
        D = torch.exp2((by - 127).double())
    else:
        e, f = by >> 3, (by & 7).double()
        D = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).double()))
        D = (D * S.double()).float().double()
    x = x.reshape(*scales.shape, n) * D.unsqueeze(-1)
    if c["rotate"]:
        x = torch.matmul(x.reshape(-1, n), _sylvester(n))
    return x.reshape(*codes.shape[:-1], -1)


def _fl32(x):
    return x.float().double()


def _exact_blocks(x, S, c):
    """What blocks x [N, n] (64 bits holding binary32 values) become in the cache, in the rotated domain."""
    n, grid = _block(c), torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def code(y):  # nearest grid value, ties to the even index
        d = (y.unsqueeze(-1) - grid).abs()
        near = d == d.amin(-1, keepdim=True)
        at = torch.arange(8, device=DEV)
        return grid[torch.where(near, at + 8 * (at & 1), 99).amin(-1) & 7]

    top = x.abs().amax(-1)
    if c["fmt"] == "mxfp4":
        D = torch.exp2((torch.floor(torch.log2(top.clamp(min=1e-300))) - 2).clamp(-127, 127))
        return torch.sign(x) * code(_fl32(x.abs() / D[:, None])) * D[:, None]
    p = torch.arange(0, 127, device=DEV)
    val = torch.where(p < 8, p.double() * 2.0 ** -9, (8 + (p & 7)).double() * torch.exp2(((p >> 3) - 10).double()))
    t = _fl32(top / _fl32(6 * S.double()))
    up = torch.bucketize(t, val).clamp(1, 126)  # the first value >= t, and the one below it
    lo = up - 1
    below, above = t - val[lo], val[up] - t
    base = torch.where((below < above) | ((below == above) & ((lo & 1) == 0)), lo, up).clamp(1, 126)
    best = D = None
    for k in range(SWEEP[0], SWEEP[1] + 1) if c["rule"] == "sweep" else (0,):
        Dk = _fl32(val[(base + k).clamp(1, 126)] * S.double())[:, None]
        err = (x.abs() - _fl32(code(_fl32(x.abs() * _fl32(1 / Dk))) * Dk)).square().sum(-1, keepdim=True)
        D = Dk if best is None else torch.where(err < best, Dk, D)
        best = err if best is None else torch.minimum(err, best)
    return torch.sign(x) * code(_fl32(x.abs() * _fl32(1 / D))) * D


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] != "attend":
        n, got = _block(c), {}
        for name in ("k", "v"):
            codes, scales, S = s[name]
            if c["op"] == "read":
                at, off = s["slots"] // c["page"], s["slots"] % c["page"]
                got[name] = _exact_values(codes[at, :, off], scales[at, :, off], S, c)
                continue
            x, parts = s[name + "_new"].float(), []
            for piece in x.reshape(-1, n).split(1 << 18):
                if c["rotate"]:
                    piece = _butterflies(piece, n)
                y = _exact_blocks(piece.double(), S, c)
                parts.append(torch.matmul(y, _sylvester(n)) if c["rotate"] else y)
            got[name] = torch.cat(parts).reshape(x.shape)
        return got
    H, G, D = c["heads"], c["group"], c["dim"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(*_lens(c))):
        if c["page"]:
            pages = s["table"][b, : -(-m // c["page"])].long()
        else:
            pages = torch.tensor([b], device=DEV)
        pos = torch.arange(m - n, m, device=DEV)[:, None]
        key = torch.arange(m, device=DEV)
        hidden = key > pos
        if c["window"]:
            hidden |= key <= pos - c["window"]
        for h in range(H):
            k, v = (_exact_values(s[x][0][pages, h].reshape(-1, D // 2)[:m], s[x][1][pages, h].reshape(-1, D // _block(c))[:m],
                                  s[x][2], c) for x in ("k", "v"))
            for j in range(h * G, h * G + G):
                w = (q[at:at + n, j] @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse[at:at + n, j] = torch.logsumexp(w, -1)
                out[at:at + n, j] = torch.softmax(w, -1) @ v
        at += n
    return {"out": out, "lse": lse}
