"""Appends of more rows than one grid, or one launch, covers, and a slot named twice. Most slots are skipped, so that the sizes cost no
memory for the cache: what counts is that each kept token lands where it belongs, turned by its own position."""
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HEADS, DIM, PAGE, PAGES = 64, 256, 16, 8


def rows_of(total, dtype, seed):
    """[total, HEADS, DIM] values of one small allocation: neighbouring rows begin 16 bytes apart."""
    step = 16 // (2 if dtype == BF16 else 4)
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = torch.randn((total + HEADS) * step + DIM, generator=g, device="cuda").to(dtype)
    return torch.as_strided(base, (total, HEADS, DIM), (step, step, 1))


@pytest.mark.parametrize("rule,dtype,fmt,lanes,with_q", [
    (B.FP4Q_SCALE_ABSMAX, BF16, B.FP4Q_NVFP4, 32, True), (B.FP4Q_SCALE_ABSMAX, F32, B.FP4Q_MXFP4, 32, False),
    (B.FP4Q_SCALE_SWEEP, BF16, B.FP4Q_NVFP4, 16, False), (B.FP4Q_SCALE_SWEEP, F32, B.FP4Q_MXFP4, 8, False)])
def test_appends_past_one_grid_and_one_launch(rule, dtype, fmt, lanes, with_q):
    """Lanes past 2^28 (2^20 workgroups of 256) and past 2^31 (a second launch); q's result, where there is one, is of 34 GB."""
    total = (1 << 31) // (HEADS * lanes) + 77
    if with_q and torch.cuda.mem_get_info()[0] < 1.2 * total * HEADS * DIM * 2:
        pytest.skip("less free memory than q takes")
    g = torch.Generator(device="cuda").manual_seed(2)
    at = torch.cat([torch.tensor([0, 1, total - 2, total - 1])] + [b + torch.arange(-2, 2) for b in
                   ((1 << 28) // (HEADS * lanes), (1 << 31) // (HEADS * lanes))] + [torch.randint(2, total - 2, (30,), generator=torch.Generator().manual_seed(1))]).unique().cuda()
    place = torch.randperm(PAGES * PAGE, generator=g, device="cuda")[:len(at)]
    slots = torch.full((total,), -1, dtype=torch.int64, device="cuda")
    slots[at] = place
    k, v = rows_of(total, dtype, 3), rows_of(total, dtype, 4)
    q = rows_of(total, dtype, 5) if with_q else None
    positions = torch.randint(0, 500, (total,), generator=g, device="cuda")
    rest = dict(rope=B.rope_table(500, 128), k_weight=torch.rand(DIM, generator=g, device="cuda") + 0.5)
    cache, want = (B.alloc_kv_cache(PAGES, HEADS, PAGE, DIM, 0.003, 0.004, format=fmt, scale_rule=rule) for _ in range(2))
    got = B.kv_append(cache, k, v, slots, q=q, positions=positions, **rest)
    few = B.kv_append(want, k[at].contiguous(), v[at].contiguous(), place, q=q[at].contiguous() if with_q else None,
                      positions=positions[at].contiguous(), **rest)
    torch.cuda.synchronize()
    for a, b in zip(cache.tensors, want.tensors):
        assert a is None or torch.equal(a, b)
    assert int((want.tensors[0] != 0).any(-1).any(1).sum()) == len(at)
    assert not with_q or torch.equal(got[at], few)


@pytest.mark.parametrize("rule", [B.FP4Q_SCALE_ABSMAX, B.FP4Q_SCALE_SWEEP])
def test_a_slot_named_twice(rule):
    """Every byte of its rows is one of the tokens', and no other row changes; q is each token's own."""
    tokens = 600
    k, v, q = (torch.randn(tokens, 2, 128, device="cuda").to(BF16) for _ in range(3))
    cache, *once = [B.alloc_kv_cache(50, 2, 16, 128, 0.003, 0.004, scale_rule=rule) for _ in range(3)]
    slots = torch.randperm(800, device="cuda")[:tokens // 2]
    both = torch.cat((slots, slots.flip(0)))
    positions, rope = torch.arange(tokens, device="cuda"), B.rope_table(tokens, 64)
    got = B.kv_append(cache, k, v, both, q=q, positions=positions, rope=rope)
    parts = [slice(i * tokens // 2, (i + 1) * tokens // 2) for i in range(2)]
    alone = [B.kv_append(c, k[p], v[p], both[p], q=q[p], positions=positions[p], rope=rope) for c, p in zip(once, parts)]
    torch.cuda.synchronize()
    for t, a, b in zip(cache.tensors, once[0].tensors, once[1].tensors):
        assert t is None or bool(((t == a) | (t == b)).all())
    assert torch.equal(got, torch.cat(alone))
