"""Writes and reads of more rows than one grid, or one launch, covers. Most slots are skipped, so that the sizes cost no
memory for the cache: what counts is that each kept token lands where it belongs."""
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

pytestmark = pytest.mark.gpu
DIM, PAGE, PAGES, KEPT = 256, 16, 64, 40


def tokens_kept(total, lanes):
    """Token numbers: the first and last ones, those around the borders of a grid's first pass and of a launch (2^28 and
    2^31 lanes), and others."""
    at = [0, 1, total - 1, total - 2]
    for b in ((1 << 28) // lanes, (1 << 31) // lanes):
        at += [b - 2, b - 1, b, b + 1]
    g = torch.Generator().manual_seed(1)
    at += torch.randint(0, total, (KEPT,), generator=g).tolist()
    at = sorted({t for t in at if 0 <= t < total})
    return torch.tensor(at)


def rows_of(total, dtype, seed):
    """[total, 1, DIM] values of one small allocation: row t begins 16 bytes behind row t - 1."""
    step = 16 // (2 if dtype == torch.bfloat16 else 4)
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = torch.empty(total * step + DIM, dtype=dtype, device="cuda")
    for part in base.split(1 << 27):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return torch.as_strided(base, (total, 1, DIM), (step, DIM, 1))


@pytest.mark.parametrize("rule,dtype,fmt,lanes", [
    (B.FP4Q_SCALE_ABSMAX, torch.bfloat16, B.FP4Q_NVFP4, 16), (B.FP4Q_SCALE_ABSMAX, torch.float32, B.FP4Q_MXFP4, 32),
    (B.FP4Q_SCALE_SWEEP, torch.bfloat16, B.FP4Q_NVFP4, 16), (B.FP4Q_SCALE_SWEEP, torch.float32, B.FP4Q_MXFP4, 8)])
@pytest.mark.parametrize("launches", [1, 2])
def test_writes_past_one_grid_and_one_launch(rule, dtype, fmt, lanes, launches):
    """One launch of more than 2^28 lanes (2^20 workgroups of 256), and lanes past 2^31 in a second launch."""
    total = (1 << 28) // lanes + 1001 if launches == 1 else (1 << 31) // lanes + 77
    at = tokens_kept(total, lanes)
    assert PAGES * PAGE >= len(at)
    g = torch.Generator(device="cuda").manual_seed(2)
    place = torch.randperm(PAGES * PAGE, generator=g, device="cuda")[:len(at)]
    slots = torch.full((total,), -1, dtype=torch.int64, device="cuda")
    slots[at.cuda()] = place
    x = [rows_of(total, dtype, s) for s in (3, 4)]
    cache, want = (B.alloc_kv_cache(PAGES, 1, PAGE, DIM, 0.003, 0.004, format=fmt, scale_rule=rule) for _ in range(2))
    B.kv_write(cache, x[0], x[1], slots)
    few = [t[at.cuda()].contiguous() for t in x]
    B.kv_write(want, few[0], few[1], place)
    torch.cuda.synchronize()
    for a, b in zip(cache.tensors, want.tensors):
        assert a is None or torch.equal(a, b)
    assert int((want.tensors[0] != 0).any(-1).sum()) == len(at)


@pytest.mark.parametrize("dtype,lanes", [(torch.float32, 64), (torch.bfloat16, 32)])
def test_reads_past_one_launch(dtype, lanes):
    """Lanes past 2^31 in a second launch; most slots are out of range and read as zeros."""
    total = (1 << 31) // lanes + 77
    room = torch.cuda.mem_get_info()[0]
    if room < 2.3 * total * DIM * (4 if dtype == torch.float32 else 2):
        pytest.skip("less free memory than the two outputs take")
    cache = B.alloc_kv_cache(PAGES, 1, PAGE, DIM, 0.003, 0.004)
    x = [torch.randn(PAGES * PAGE, 1, DIM, device="cuda") for _ in range(2)]
    B.kv_write(cache, x[0], x[1], torch.arange(PAGES * PAGE, device="cuda"))
    at = tokens_kept(total, lanes).cuda()
    place = torch.arange(len(at), device="cuda") * 3 + 1
    slots = torch.full((total,), PAGES * PAGE, dtype=torch.int64, device="cuda")
    slots[at] = place
    got = B.kv_read(cache, slots, dtype=dtype)
    want = B.kv_read(cache, place, dtype=dtype)
    for a, b in zip(got, want):
        assert torch.equal(a[at], b)
        assert int((b != 0).any(-1).sum()) == len(at)
        a[at] = 0
        assert not any(bool(p.any()) for p in a.split(1 << 22))


@pytest.mark.parametrize("fmt", [B.FP4Q_NVFP4, B.FP4Q_MXFP4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_slot_named_twice(fmt, dtype):
    """Every byte of its rows is one of the tokens', and no other row changes."""
    tokens = 600
    x = [torch.randn(tokens, 2, 128, device="cuda").to(dtype) for _ in range(2)]
    once = [B.alloc_kv_cache(50, 2, 16, 128, 0.003, 0.004, format=fmt) for _ in range(2)]
    cache = B.alloc_kv_cache(50, 2, 16, 128, 0.003, 0.004, format=fmt)
    slots = torch.randperm(800, device="cuda")[:tokens // 2]
    both = torch.cat((slots, slots.flip(0)))
    B.kv_write(cache, x[0], x[1], both)
    for i in range(2):
        part = slice(i * tokens // 2, (i + 1) * tokens // 2)
        B.kv_write(once[i], x[0][part], x[1][part], both[part])
    torch.cuda.synchronize()
    for got, a, b in zip(cache.tensors, once[0].tensors, once[1].tensors):
        assert got is None or bool(((got == a) | (got == b)).all())
    k, v = B.kv_read(cache, slots)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
