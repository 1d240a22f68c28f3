"""Products on other streams, with workspaces of the caller's that hold anything before, and in replayed graphs, against 64 bits."""
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from test_gpu_matmul_forms import F32, F64, HALF, block_of, sums, weight

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
# format, type of x, rotated, rows of the weight, columns, rows of x: prepared x of few rows, of many, partial sums, both, neither
CALLS = [("nvfp4", F32, False, 37, 1536, 13), ("mxfp4", BF16, True, 301, 288, 40), ("nvfp4", BF16, False, 301, 1024, 65),
         ("mxfp4", F32, False, 515, 2048, 100), ("nvfp4", BF16, True, 515, 2592, 3001), ("mxfp4", BF16, False, 37, 800, 3)]


class Call:
    def __init__(self, case, seed):
        self.fmt, self.dtype, self.rotate, n, k, m = case
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w, self.v = weight(gen, self.fmt, n, k, self.rotate)
        self.x = torch.randn(m, k, device="cuda", generator=gen).to(self.dtype)
        self.need = B.matmul_workspace_bytes(self.w, m, self.dtype)

    def check(self, got):
        parts = 1 if self.dtype == BF16 and not self.rotate else 3
        y, tol = sums(self.x.to(F64), self.v, block_of(self.fmt), self.rotate, parts)
        off = (got.to(F64) - y).abs()
        assert (off <= tol + HALF[self.dtype] * (y.abs() + tol) + 1e-37).all()


@pytest.mark.parametrize("case", CALLS, ids=str)
def test_workspaces_that_hold_anything(case):
    """NaN patterns, then what another call left; what lies behind the workspace stays."""
    call = Call(case, 1)
    space = torch.full((call.need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    call.check(B.matmul(call.w, call.x, workspace=space[:call.need]))
    assert (space[call.need:] == 0xFF).all()
    call.x = call.x.flip(0).contiguous() * 3
    call.check(B.matmul(call.w, call.x, workspace=space))
    assert (space[call.need:] == 0xFF).all()
    if call.need:
        with pytest.raises(ValueError):
            B.matmul(call.w, call.x, workspace=space[:call.need - 1])


@pytest.mark.parametrize("case", CALLS, ids=str)
def test_two_streams_at_once(case):
    calls = [Call(case, 1), Call(case, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            got[i].append(B.matmul(calls[i].w, calls[i].x, stream=s))
    torch.cuda.synchronize()
    for call, ys in zip(calls, got):
        for y in ys:
            call.check(y)
            assert torch.equal(y, ys[0])


@pytest.mark.parametrize("case", CALLS, ids=str)
def test_replayed_graphs(case):
    """x and what the workspace held change between replays, with eager work in between."""
    call = Call(case, 3)
    space = torch.empty(max(call.need, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty(call.x.shape[0], call.w.rows, dtype=call.dtype, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    B.matmul(call.w, call.x, out=out, workspace=space)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        B.matmul(call.w, call.x, out=out, workspace=space)
    for i in range(4):
        call.x.copy_(torch.randn(call.x.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(10 + i)))
        space.fill_(0xFF)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        call.check(out)
        assert torch.equal(out, B.matmul(call.w, call.x))
