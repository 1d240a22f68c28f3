"""A layer with 4-bit weights and a 4-bit cache: the projections, the append, attention, the gated block, run together for a
prompt and for single tokens, each step against 64 bits on what the step before gave; and the same captured and
replayed, on other streams, with workspaces that hold anything."""
import math

import numpy as np
import pytest
import torch

from append_common import bytes_of, turned
from block_scaled_fp4_fp4q_amd import binding as B
from matmul_common import Made, close, product64, rounded
from test_gpu_matmul import gated64

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Layer:
    H, G, D, W, F = 2, 3, 64, 256, 480  # KV heads, queries of each, head size, width, inner width

    def __init__(self, fmt, rotate, pages=12, page=16):
        rng = np.random.default_rng(7)
        n_qkv = self.H * (self.G + 2) * self.D
        self.made = {k: Made(rng, fmt, n, w, rotate, S) for k, n, w, S in (
            ("qkv", n_qkv, self.W, 0.004), ("o", self.W, self.H * self.G * self.D, 0.004), ("gate", self.F, self.W, 0.003),
            ("up", self.F, self.W, 0.003), ("down", self.W, self.F, 0.003))}
        self.w = {k: m.handle() for k, m in self.made.items()}
        self.fmt, self.rotate, self.page = fmt, rotate, page
        self.S = (np.float32(0.01), np.float32(0.02))
        f, _, block = (B.FP4Q_NVFP4, 0, 16) if fmt == "nvfp4" else (B.FP4Q_MXFP4, 1, 32)
        self.cache = B.alloc_kv_cache(pages, self.H, page, self.D, *self.S, format=f, rotate=block if rotate else 0)
        self.qw, self.kw = [(1 + 0.2 * rng.standard_normal(self.D)).astype(np.float32) for _ in range(2)]
        self.dqw, self.dkw = torch.from_numpy(self.qw).cuda(), torch.from_numpy(self.kw).cuda()
        self.rope = B.rope_table(400, 32, base=1000.0)

    def run(self, x, slots, positions, kv_lens, table, max_kv, starts=None, max_q=None):
        r = {}
        t = x.shape[0]
        r["qkv"] = B.matmul(self.w["qkv"], x)
        rows = r["qkv"].view(t, -1, self.D)
        hq = self.H * self.G
        r["q"] = B.kv_append(self.cache, rows[:, hq:hq + self.H], rows[:, hq + self.H:], slots, q=rows[:, :hq], positions=positions,
                             rope=self.rope, q_weight=self.dqw, k_weight=self.dkw, eps=1e-6)
        r["a"] = B.attend(self.cache, r["q"], kv_lens, max_kv=max_kv, block_table=table, q_starts=starts, max_q=max_q)
        r["o"] = B.matmul(self.w["o"], r["a"].view(t, -1))
        r["g"] = B.gated(self.w["gate"], self.w["up"], r["o"])
        r["y"] = B.matmul(self.w["down"], r["g"])
        return r

    def check(self, x, r, slots, positions, seen):
        """seen(i): the slots that query row i attends to, in order."""
        def product(name, of, got):
            y, tol = product64(self.made[name], of.cpu())
            close(got, y, rounded(y, tol, BF16))

        product("qkv", x, r["qkv"])
        rows = r["qkv"].float().cpu().numpy().reshape(x.shape[0], -1, self.D)
        hq = self.H * self.G
        table = self.rope.cpu().numpy()
        q = turned(rows[:, :hq], self.qw, 1e-6, table, positions, False)
        assert torch.equal(r["q"].cpu(), torch.from_numpy(q).to(BF16))
        new = (turned(rows[:, hq:hq + self.H], self.kw, 1e-6, table, positions, False), rows[:, hq + self.H:])
        for side in range(2):
            for i, want in enumerate(bytes_of(new[side], self.fmt, "absmax", self.S[side], self.rotate)):
                got = self.cache.tensors[3 * side + i].cpu().numpy()[slots // self.page, :, slots % self.page]
                assert np.array_equal(got, want)
        q = r["q"].double().cpu().numpy()
        for i in range(x.shape[0]):
            k, v = (t.double().cpu().numpy() for t in B.kv_read(self.cache, torch.from_numpy(seen(i)).cuda()))
            for h in range(hq):
                s = k[:, h // self.G] @ q[i, h] / math.sqrt(self.D)
                p = np.exp(s - s.max())
                p /= p.sum()
                o, size = p @ v[:, h // self.G], p @ np.abs(v[:, h // self.G])
                # the result's rounding, probabilities in 11 bits at least, logits to 2^-16 or so of theirs; where rows
                # are stored rotated, the binary32 sums of the transform of a block, here and in kv_read
                tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * size
                if self.rotate:
                    n = self.made["o"].block
                    tol += 2 * (n + 2) * 2.0 ** -24 * np.repeat(size.reshape(-1, n).sum(-1), n)
                bad = np.abs(r["a"][i, h].double().cpu().numpy() - o) > tol
                assert not bad.any(), (i, h, np.flatnonzero(bad)[:4])
        product("o", r["a"].view(x.shape[0], -1), r["o"])
        y, tol = gated64(self.made["gate"], self.made["up"], r["o"].cpu(), B.FP4Q_ACT_SILU)
        close(r["g"], y, rounded(y, tol, BF16))
        product("down", r["g"], r["y"])


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_prompt_then_tokens(fmt, rotate):
    rng = np.random.default_rng(3)
    layer = Layer(fmt, rotate)
    lens = [37, 21]
    table = torch.tensor([[3, 7, 0, 5], [9, 1, 4, 11]], dtype=torch.int32, device="cuda")
    slot = lambda b, t: int(table[b, t // 16]) * 16 + t % 16  # noqa: E731
    where = [(b, t) for b in range(2) for t in range(lens[b])]
    make = lambda n: torch.from_numpy(rng.standard_normal((n, layer.W)).astype(np.float32)).to(BF16).cuda()  # noqa: E731
    dev = lambda x, d: torch.tensor(x, dtype=d, device="cuda")  # noqa: E731

    def go(where, lens, **kw):
        slots, pos = np.array([slot(b, t) for b, t in where]), np.array([t for _, t in where])
        x = make(len(where))
        r = layer.run(x, dev(slots, torch.int64), dev(pos, torch.int64), dev(lens, torch.int32), table, 64, **kw)
        layer.check(x, r, slots, pos, lambda i: np.array([slot(where[i][0], t) for t in range(where[i][1] + 1)]))

    go(where, lens, starts=dev([0, 37, 58], torch.int32), max_q=37)
    for _ in range(3):
        where = [(b, lens[b]) for b in range(2)]
        lens = [n + 1 for n in lens]
        go(where, lens)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("tokens", [2, 90])
def test_captured_and_replayed(tokens, rotate):
    """The whole layer in one graph: replays, with other inputs, eager work on other data and synchronizations between
    them, give the eager results."""
    layer = Layer("nvfp4", rotate)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, layer.W, generator=g, device="cuda").to(BF16)
    slots = torch.randperm(12 * 16, generator=g, device="cuda")[:tokens]
    pos = torch.randint(0, 400, (tokens,), generator=g, device="cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda")[None].repeat(tokens, 1)
    lens = torch.full((tokens,), 150, dtype=torch.int32, device="cuda")
    for t in layer.cache.tensors[:2] + layer.cache.tensors[3:5]:  # a cache with something in it
        t.copy_(torch.randint(0, 0x70, t.shape, generator=g, device="cuda").to(torch.uint8))
    args = (slots, pos, lens, table, 192)
    start = [t.clone() for t in (layer.cache.tensors[i] for i in (0, 1, 3, 4))]

    def reset():
        for t, s in zip((layer.cache.tensors[i] for i in (0, 1, 3, 4)), start):
            t.copy_(s)

    layer.run(x, *args)
    graph = torch.cuda.CUDAGraph()
    reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = layer.run(x, *args)
    for seed in range(4):
        x.copy_(torch.randn(tokens, layer.W, generator=g, device="cuda"))
        reset()
        eager = {k: v.clone() for k, v in layer.run(x, *args).items()}
        held = [layer.cache.tensors[i].clone() for i in (0, 1, 3, 4)]
        reset()
        for v in out.values():
            v.zero_()
        if seed % 2:
            torch.cuda.synchronize()
        graph.replay()
        other = torch.randn(300, layer.W, device="cuda").to(BF16)  # eager work beside it
        B.matmul(layer.w["up"], other)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(torch.nan_to_num(out[k].float(), 9.0), torch.nan_to_num(eager[k].float(), 9.0)), k
        assert all(torch.equal(layer.cache.tensors[i], h) for i, h in zip((0, 1, 3, 4), held))


def test_streams_and_workspaces():
    """Two calls at once on two streams with workspaces of their own, filled with NaN bits, on a stream that is not the
    current one; the results are those of calls alone."""
    rng = np.random.default_rng(2)
    made = [Made(rng, f, 300, 2048, True) for f in ("nvfp4", "mxfp4")]
    ws = [m.handle() for m in made]
    xs = [torch.from_numpy(rng.standard_normal((m, 2048)).astype(np.float32)).cuda() for m in (70, 23)]
    alone = [B.matmul(w, x) for w, x in zip(ws, xs)]
    both = [B.gated(w, w, x) for w, x in zip(ws, xs)]
    need = [max(B.matmul_workspace_bytes(w, x.shape[0], x.dtype), B.gated_workspace_bytes(w, w, x.shape[0], x.dtype))
            for w, x in zip(ws, xs)]
    spaces = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in need]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [B.matmul(w, x, workspace=p, stream=s) for w, x, p, s in zip(ws, xs, spaces, streams)]
        two = [B.gated(w, w, x, workspace=p, stream=s) for w, x, p, s in zip(ws, xs, spaces, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone)) and all(torch.equal(a, b) for a, b in zip(two, both))
    with pytest.raises(ValueError):
        B.matmul(ws[0], xs[0], workspace=spaces[0][:100])
    short = B.matmul_workspace_bytes(ws[0], 70, torch.float32)
    exact = torch.full((short + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    assert torch.equal(B.matmul(ws[0], xs[0], workspace=exact[:short]), alone[0])
    assert (exact[short:] == 0x5A).all()  # nothing past what was asked for
