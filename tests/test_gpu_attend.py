"""Attention over the 4-bit KV cache against the formula in 64 bits, within bounds that follow the arithmetic."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import Filled, attention64, check

pytestmark = pytest.mark.gpu


def queries(rng, total, heads, dim, dtype, size=1.0):
    q = torch.from_numpy((size * rng.standard_normal((total, heads, dim))).astype(np.float32))
    return q.to(torch.bfloat16) if dtype == "bf16" else q


def starts_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def run(f, q, q_lens, causal=True, window=0, scale=None, what="", uniform=False, cache=None, **kw):
    st = starts_of(q_lens)
    want = attention64(f, q.double().numpy(), st, causal, window, scale, q.dtype == torch.bfloat16)
    out, lse = B.attend(cache or f.cache(), q.cuda(), torch.tensor(f.lens, dtype=torch.int32, device="cuda"),
                        block_table=f.device_table(), causal=causal, window=window, scale=scale, return_lse=True,
                        q_starts=None if uniform else torch.from_numpy(st).cuda(),
                        **({} if uniform else {"max_q": max(q_lens)}), **kw)
    torch.cuda.synchronize()
    check(out, lse, *want, what=what)
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_single_tokens(fmt, dim, rotate, dtype):
    """One query per sequence, lengths around the tiles of 16, 32 and 128 keys and the chunks."""
    rng = np.random.default_rng(21)
    lens = [1, 15, 16, 17, 31, 33, 127, 129, 300, 0]
    f = Filled(rng, fmt, dim, 2, 16, lens, rotate)
    run(f, queries(rng, len(lens), 2 * 4, dim, dtype), [1] * len(lens), uniform=True, what=f"{fmt} {dim}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_packed_prompts(fmt, dim, rotate, dtype):
    """Prompts of different lengths one after another, some after a prefix; one has more queries than keys."""
    rng = np.random.default_rng(22)
    q_lens, lens = [1, 70, 33, 130, 16, 9], [5, 70, 133, 130, 400, 4]
    f = Filled(rng, fmt, dim, 2, 32, lens, rotate)
    run(f, queries(rng, sum(q_lens), 2 * 3, dim, dtype), q_lens, what=f"{fmt} {dim}")


@pytest.mark.parametrize("group", [1, 2, 5, 7, 16, 17, 40, 71])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_groups(fmt, group):
    rng = np.random.default_rng(23)
    lens, q_lens = [50, 131, 3], [2, 5, 1]
    f = Filled(rng, fmt, 128, 3, 16, lens)
    run(f, queries(rng, sum(q_lens), 3 * group, 128, "bf16"), q_lens, what=f"group {group}")


@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 1000])
@pytest.mark.parametrize("q_len", [1, 4, 90])
def test_windows(q_len, window):
    rng = np.random.default_rng(24)
    lens = [q_len, q_len + 29, q_len + 257, q_len + 700]
    f = Filled(rng, "nvfp4", 64, 2, 16, lens)
    run(f, queries(rng, 4 * q_len, 4, 64, "bf16"), [q_len] * 4, window=window, what=f"window {window}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("q_lens", [[3, 3, 3], [100, 7, 40]])
def test_every_key_seen(fmt, q_lens):
    rng = np.random.default_rng(25)
    f = Filled(rng, fmt, 128, 2, 48, [200, 1, 65])
    run(f, queries(rng, sum(q_lens), 4, 128, "bf16"), q_lens, causal=False)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
@pytest.mark.parametrize("contiguous,page", [(True, 333), (True, 64), (False, 16), (False, 48), (False, 512)])
def test_layouts_and_pages(contiguous, page, layout):
    """Pages that end inside a tile, caches without pages whose length is no multiple of anything, orders of the
    dimensions; NaN scales stand behind every sequence's last row."""
    rng = np.random.default_rng(26)
    lens = [333, 200, 1] if page == 333 else [64, 63, 33] if contiguous else [333, 200, 1]
    f = Filled(rng, "nvfp4", 128, 3, page, lens, contiguous=contiguous, layout=layout)
    for q_lens in ([1, 1, 1], [30, 64 if page != 64 else 33, 1]):
        run(f, queries(rng, sum(q_lens), 6, 128, "bf16"), q_lens, what=f"{layout} {page}")


def test_strided_queries_and_outputs():
    rng = np.random.default_rng(27)
    f = Filled(rng, "nvfp4", 128, 2, 16, [40, 90])
    for q_lens in ([1, 1], [40, 70]):
        total = sum(q_lens)
        q = queries(rng, total, 6, 128, "bf16")
        wide = torch.zeros(6, total, 3 * 128, dtype=torch.bfloat16, device="cuda")
        wide[:, :, 128:256] = q.cuda().transpose(0, 1)
        qv = wide[:, :, 128:256].transpose(0, 1)
        big = torch.full((6, total, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        st = starts_of(q_lens)
        want = attention64(f, q.double().numpy(), st)
        out, lse = B.attend(f.cache(), qv, torch.tensor(f.lens, dtype=torch.int32, device="cuda"), block_table=f.device_table(),
                            q_starts=torch.from_numpy(st).cuda(), max_q=max(q_lens), return_lse=True,
                            out=big[:, :, :128].transpose(0, 1))
        check(out, lse, *want)
        assert torch.all(big[:, :, 128:] == 7.0)


def test_rows_of_no_sequence_stay():
    """Rows before the first, behind the last sequence and of a sequence whose starts run backwards or too far."""
    rng = np.random.default_rng(28)
    f = Filled(rng, "nvfp4", 64, 1, 16, [20, 20, 20])
    q = queries(rng, 12, 2, 64, "bf16").cuda()
    for starts, written in (([2, 4, 6, 8], range(2, 8)), ([0, 5, 3, 6], list(range(0, 6))), ([0, 2, 13, 14], range(0, 2)),
                            ([-1, 2, 4, 6], range(2, 6))):
        out = torch.full((12, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        B.attend(f.cache(), q, torch.tensor(f.lens, dtype=torch.int32, device="cuda"), block_table=f.device_table(),
                 q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), max_q=6, out=out)
        same = [bool(torch.all(out[r] == 3.0)) for r in range(12)]
        assert same == [r not in written for r in range(12)], (starts, same)


@pytest.mark.parametrize("q_len", [1, 3, 80])
def test_bad_lengths_and_pages_give_nan(q_len):
    rng = np.random.default_rng(29)
    lens = [100, 100, 100, 100, 100]
    f = Filled(rng, "nvfp4", 128, 2, 16, lens)
    q = queries(rng, 5 * q_len, 4, 128, "bf16")
    st = starts_of([q_len] * 5)
    want, wlse, tol, ltol, own = attention64(f, q.double().numpy(), st)
    table = f.device_table().clone()
    table[2, 5] = 1 << 30
    table[3, 0] = -1
    kv = torch.tensor([100, -1, 100, 100, 113], dtype=torch.int32, device="cuda")
    out, lse = B.attend(f.cache(), q.cuda(), kv, block_table=table, max_kv=112, return_lse=True)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    bad = np.zeros((5, q_len), bool)
    bad[1] = bad[4] = bad[3] = True
    bad[2] = np.arange(q_len) + 100 - q_len >= 80  # those that see a key of page 5
    bad = bad.reshape(-1)
    assert np.all(np.isnan(out[bad])) and np.all(np.isnan(lse[bad]))
    assert np.all(np.abs(out[~bad] - want[~bad]) <= tol[~bad])


def test_pages_that_no_query_sees_are_not_looked_at():
    rng = np.random.default_rng(30)
    f = Filled(rng, "nvfp4", 128, 2, 16, [300, 260])
    q = queries(rng, 2, 4, 128, "bf16")
    want = attention64(f, q.double().numpy(), starts_of([1, 1]), window=40)
    f.table[0, :(300 - 40) // 16] = -1
    f.table[1, :(260 - 40) // 16] = -5
    out, lse = B.attend(f.cache(), q.cuda(), torch.tensor(f.lens, dtype=torch.int32, device="cuda"),
                        block_table=f.device_table(), window=40, return_lse=True)
    check(out, lse, *want)


@pytest.mark.parametrize("size", [1e-30, 30.0, 1e4])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes_of_queries(fmt, dtype, size):
    """Queries so small that all keys count alike, and so large that one key alone does."""
    rng = np.random.default_rng(31)
    f = Filled(rng, fmt, 128, 2, 16, [150, 77])
    run(f, queries(rng, 2, 4, 128, dtype, size), [1, 1], what=f"size {size}")
    run(f, queries(rng, 100, 4, 128, dtype, size), [60, 40], what=f"size {size}")


def test_infinite_and_nan_queries_stay_in_their_rows():
    rng = np.random.default_rng(32)
    f = Filled(rng, "nvfp4", 128, 1, 16, [90])
    for n in (3, 70):
        q = queries(rng, n, 2, 128, "bf16")
        want, wlse, tol, ltol, own = attention64(f, q.double().numpy(), starts_of([n]))
        q[1, 0, 5] = float("nan")
        q[2, 1, 7] = float("inf")
        out, _ = B.attend(f.cache(), q.cuda(), torch.tensor([90], dtype=torch.int32, device="cuda"),
                          block_table=f.device_table(), return_lse=True)
        out = out.float().cpu().numpy()
        assert np.all(np.isnan(out[1, 0])) and np.all(np.isnan(out[2, 1]))
        keep = np.ones((n, 2), bool)
        keep[1, 0] = keep[2, 1] = False
        assert np.all(np.abs(out - want)[keep] <= tol[keep])


def test_long_contexts_split_over_workgroups():
    rng = np.random.default_rng(33)
    f = Filled(rng, "nvfp4", 64, 1, 64, [9001, 40, 5000], rotate=True)
    run(f, queries(rng, 3, 2, 64, "bf16"), [1, 1, 1], uniform=True)
    run(f, queries(rng, 12, 2, 64, "f32"), [4, 4, 4], uniform=True)
    q_lens = [90, 10, 33]
    run(f, queries(rng, sum(q_lens), 2, 64, "bf16"), q_lens)


@pytest.mark.parametrize("batch", [64, 65, 130, 256, 257, 700])
def test_many_sequences(batch):
    """Lengths of many sequences, most short, a few long, some empty: those that a workgroup looks through itself and
    those that are written down first."""
    rng = np.random.default_rng(37)
    lens = [int(n) for n in rng.integers(0, 60, batch)]
    for b in rng.integers(0, batch, 5):
        lens[b] = int(rng.integers(500, 3000))
    f = Filled(rng, "nvfp4", 64, 2, 16, lens)
    run(f, queries(rng, batch, 4, 64, "bf16"), [1] * batch, uniform=True, what=f"batch {batch}")
    q_lens = [int(n) for n in rng.integers(0, 4, batch)]
    run(f, queries(rng, sum(q_lens), 4, 64, "bf16"), q_lens, what=f"batch {batch}, packed")


def test_cache_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes whose used pages lie at its end."""
    rng = np.random.default_rng(34)
    f = Filled(rng, "nvfp4", 256, 2, 16, [70], spare=0)
    pages = (1 << 32) // (2 * 16 * 128) + 100
    big = torch.empty(pages, 2, 16, 128, dtype=torch.uint8, device="cuda")
    small = f.cache()
    used = len(f.codes[0])
    kc, ks, kg, vc, vs, vg = small.tensors
    scales = [torch.empty(pages, 2, 16, 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    big[-used:], scales[0][-used:], scales[1][-used:] = kc, ks, vs
    cache = B.KvCache(big, scales[0], kg, big, scales[1], vg)
    f.table += pages - used
    f.kv[0][1] = None  # V has K's codes: redo its values
    from oracle import ref
    got = f.table[0] - (pages - used)
    c = np.concatenate([f.codes[0][p] for p in got], 1)[:, :70]
    s = np.concatenate([f.scales[1][p] for p in got], 1)[:, :70]
    f.kv[0][1] = ref.dequantize(np.ascontiguousarray(c), np.ascontiguousarray(s), float(f.S[1]), 140, 256).reshape(2, 70, 256).astype(np.float64)
    for q_lens in ([1], [70]):
        run(f, queries(rng, q_lens[0], 4, 256, "bf16"), q_lens, cache=cache)
    del big, scales, cache


def test_other_stream_and_given_workspace():
    rng = np.random.default_rng(35)
    f = Filled(rng, "nvfp4", 128, 2, 16, [2000, 900])
    q = queries(rng, 2, 8, 128, "bf16")
    want = attention64(f, q.double().numpy(), starts_of([1, 1]))
    cache, table = f.cache(), f.device_table()
    lens = torch.tensor(f.lens, dtype=torch.int32, device="cuda")
    qd = q.cuda()
    need = B.attend_workspace_bytes(cache, qd, lens, block_table=table)
    assert need > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for turn in range(6):  # two streams at once, each with its own workspace
        s = streams[turn % 2]
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        got.append((B.attend(cache, qd, lens, block_table=table, return_lse=True, workspace=ws, stream=s), ws))
        got.append((B.attend(cache, qd, lens, block_table=table, return_lse=True, stream=s), None))
    torch.cuda.synchronize()
    for (out, lse), _ in got:
        check(out, lse, *want)
        assert torch.equal(out, got[0][0][0]) and torch.equal(lse, got[0][0][1])  # no order of sums that varies


def test_captured_steps_replay():
    """A decode step (write the new token, attend) captured once and replayed with other inputs, with eager calls and
    synchronizations between; two graphs, each with its own workspace."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(5)
    heads, group, dim, page, batch = 2, 4, 128, 16, 3
    caches = [B.alloc_kv_cache(60, heads, page, dim, 0.01, 0.01, rotate=16, scale_rule=B.FP4Q_SCALE_SWEEP)
              for _ in range(2)]
    table = torch.randperm(60, generator=g, device=dev).to(torch.int32).reshape(batch, 20)
    new = [torch.zeros(batch, heads, dim, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    q = torch.zeros(batch, heads * group, dim, dtype=torch.bfloat16, device=dev)
    lens = torch.ones(batch, dtype=torch.int32, device=dev)
    slots = torch.zeros(batch, dtype=torch.int64, device=dev)
    outs = [torch.zeros_like(q) for _ in range(2)]
    need = B.attend_workspace_bytes(caches[0], q, lens, block_table=table)
    spaces = [torch.empty(max(need, 1), dtype=torch.uint8, device=dev) for _ in range(2)]

    def step(cache, out, ws):
        B.kv_write(cache, new[0], new[1], slots)
        B.attend(cache, q, lens, block_table=table, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[1], outs[1], spaces[1])
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(caches[0], outs[i], spaces[i])
        graphs.append(graph)
    for at in range(40):
        new[0].copy_(torch.randn(new[0].shape, generator=g, device=dev))
        new[1].copy_(torch.randn(new[0].shape, generator=g, device=dev))
        q.copy_(torch.randn(q.shape, generator=g, device=dev))
        lens.fill_(at + 1)
        slots.copy_(table[:, at // page].long() * page + at % page)
        graphs[at % 2].replay()
        eager = torch.zeros_like(q)
        step(caches[1], eager, spaces[1 - at % 2])
        torch.cuda.synchronize()
        assert torch.equal(outs[at % 2], eager), at


def test_a_serving_run():
    """Prompts written and attended, then tokens one at a time: every step against the 64-bit formula over the values
    that the cache reads back."""
    rng = np.random.default_rng(36)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(6)
    heads, group, dim, page = 2, 2, 64, 16
    prompts = [37, 5, 64]
    cache = B.alloc_kv_cache(40, heads, page, dim, 0.004, 0.004, rotate=16, scale_rule=B.FP4Q_SCALE_SWEEP)
    table = torch.from_numpy(rng.permutation(40)[:24].reshape(3, 8).astype(np.int32)).to(dev)
    have = [0, 0, 0]

    class Seen:
        pass

    for step in range(6):
        n = prompts if step == 0 else [1, 1, 1]
        total = sum(n)
        slots = torch.cat([table[b, (have[b] + torch.arange(n[b], device=dev)) // page].long() * page +
                           (have[b] + torch.arange(n[b], device=dev)) % page for b in range(3)])
        k, v = (torch.randn(total, heads, dim, generator=g, device=dev).bfloat16() for _ in range(2))
        B.kv_write(cache, k, v, slots)
        have = [h + m for h, m in zip(have, n)]
        q = torch.randn(total, heads * group, dim, generator=g, device=dev).bfloat16()
        lens = torch.tensor(have, dtype=torch.int32, device=dev)
        st = starts_of(n)
        out, lse = B.attend(cache, q, lens, block_table=table, q_starts=torch.from_numpy(st).to(dev), max_q=max(n),
                            return_lse=True)
        f = Seen()
        f.fmt, f.heads, f.lens, f.rotate, f.kv = "nvfp4", heads, have, 0, []
        for b in range(3):
            at = torch.arange(have[b], device=dev)
            got = B.kv_read(cache, table[b, at // page].long() * page + at % page)
            f.kv.append([t.double().cpu().numpy().transpose(1, 0, 2) for t in got])
        want, wlse, tol, ltol, own = attention64(f, q.double().cpu().numpy(), st)
        # the rows here are read back un-rotated, each value off by up to (16 + 2) half steps of binary32 of its
        # block's values; the attention's bound grows by as much of sum p |v| <= max |v|, and by the logits' share
        big = max(float(np.abs(x).max()) for s in f.kv for x in s)
        slack = 64 * 2.0 ** -24 * big * (1 + 8 * dim ** 0.5 * big)
        check(out, lse, want, wlse, tol + slack, ltol + slack, own, what=f"step {step}")
