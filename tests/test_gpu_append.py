"""New tokens into the 4-bit KV cache with norm and rotary positions: q bit for bit against the definition's binary32 steps, every byte of
the cache against the oracle's bytes of those rows."""
import numpy as np
import pytest
import torch

from append_common import FMT, RULE, as_type, bytes_of, turned
from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import values

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def same(got, want):
    return torch.equal(torch.nan_to_num(got.float().cpu(), 12345.0), torch.nan_to_num(want.float(), 12345.0))


class Case:
    """Inputs on the host, what they give, and the call."""

    def __init__(self, seed, fmt="nvfp4", rule="absmax", dtype=BF16, rotate=False, tokens=13, heads=2, group=3, dim=128, page=16,
                 turn=128, interleaved=False, norm=True, window=None, drop=(), lost=(), reach=77):
        rng = np.random.default_rng(seed)
        self.__dict__.update(locals())
        rows = lambda h: as_type(values(rng, (tokens, h, dim)), dtype)  # noqa: E731
        self.q, self.k, self.v = rows(heads * group), rows(heads), rows(heads)
        self.qw, self.kw = [(1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) if norm else None for _ in range(2)]
        angle = np.arange(reach)[:, None] * 100.0 ** (-np.arange(turn // 2) / max(1, turn // 2))
        self.table = np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32) if turn else None
        self.positions = rng.integers(0, reach, tokens)
        self.pages = -(-tokens // page) + 2
        self.slots = rng.permutation(self.pages * page)[:tokens]
        for i, bad in drop:
            self.slots[i] = bad if bad < 0 else self.pages * page + bad
        for i, bad in lost:
            self.positions[i] = bad if bad < 0 else reach + bad
        self.S = (np.float32(0.013), np.float32(0.021))
        self.eps = 1e-5

    def expected(self):
        args = (self.eps, self.table, self.positions, self.interleaved)
        q = turned(self.q.float().numpy(), self.qw, *args)
        k = turned(self.k.float().numpy(), self.kw, *args)
        good = (self.slots >= 0) & (self.slots < self.pages * self.page)
        if self.table is not None:
            good &= (self.positions >= 0) & (self.positions < self.reach)
        sides = [bytes_of(np.nan_to_num(x), self.fmt, self.rule, S, self.rotate, self.window)
                 for x, S in zip((k, self.v.float().numpy()), self.S)]
        return as_type(q, self.dtype), sides, good

    def cache(self):
        f, _, block = FMT[self.fmt]
        c = B.alloc_kv_cache(self.pages, self.heads, self.page, self.dim, *self.S, format=f, scale_rule=RULE[self.rule][0],
                             window=self.window, rotate=block if self.rotate else 0)
        for t in (c.tensors[0], c.tensors[1], c.tensors[3], c.tensors[4]):
            t.fill_(0xA5)
        return c

    def call(self, cache, **kw):
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        a = dict(q=self.q.cuda(), positions=dev(self.positions), rope=dev(self.table), interleaved=self.interleaved,
                 q_weight=dev(self.qw), k_weight=dev(self.kw), eps=self.eps)
        a.update(kw)
        k, v, slots = (a.pop(n, d) for n, d in (("k", self.k.cuda()), ("v", self.v.cuda()), ("slots", dev(self.slots))))
        return B.kv_append(cache, k, v, slots, **a)

    def check_cache(self, cache, sides, good):
        at = self.slots[good]
        for side, name in enumerate("kv"):
            for i, what in enumerate(("codes", "scales")):
                t, w = cache.tensors[3 * side + i].cpu().numpy(), sides[side][i]
                full = np.full(t.shape, 0xA5, np.uint8)
                full[at // self.page, :, at % self.page] = w[good]
                assert np.array_equal(t, full), f"{what} of {name}: {np.sum(t != full)} bytes differ"

    def check(self, **kw):
        cache = self.cache()
        got = self.call(cache, **kw)
        q, sides, good = self.expected()
        assert same(got, q), f"q: {(got.float().cpu() != q.float()).sum()} values differ"
        self.check_cache(cache, sides, good)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("fmt,rule,window", [("nvfp4", "absmax", None), ("nvfp4", "sweep", None), ("nvfp4", "sweep", (-1, 2)),
                                             ("nvfp4", "foursix", None), ("mxfp4", "absmax", None), ("mxfp4", "sweep", None)])
def test_rules(fmt, rule, window, rotate, dtype):
    Case(3, fmt, rule, dtype, rotate, window=window).check()


@pytest.mark.parametrize("rule", ["absmax", "sweep"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,turn", [(64, 64), (64, 16), (64, 48), (128, 0), (128, 16), (128, 96), (128, 112), (256, 256), (256, 80)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_turned_parts_of_heads(fmt, dim, turn, interleaved, rule):
    """Pairs across lanes and blocks, and inside them; a part of the head, and none of it."""
    Case(dim + turn, fmt, rule, dim=dim, turn=turn, interleaved=interleaved, rotate=turn % 32 == 0).check()


@pytest.mark.parametrize("tokens,heads,group", [(1, 1, 1), (1, 8, 5), (2, 3, 7), (64, 1, 16), (257, 4, 2), (1003, 2, 1)])
def test_numbers_of_rows(tokens, heads, group):
    Case(tokens, tokens=tokens, heads=heads, group=group, reach=5000, page=48).check()


@pytest.mark.parametrize("norm_q,norm_k", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rule", ["absmax", "sweep"])
def test_without_norms(norm_q, norm_k, rule):
    c = Case(9, rule=rule, rotate=True)
    c.qw, c.kw = c.qw if norm_q else None, c.kw if norm_k else None
    c.check()


def test_without_q():
    c = Case(10)
    cache = c.cache()
    assert c.call(cache, q=None) is None
    c.check_cache(cache, *c.expected()[1:])


def test_plain_rows_are_those_of_a_write():
    """Without norm and positions the cache holds what kv_write puts there, and q is handed on."""
    c = Case(12, "mxfp4", "sweep", F32, True, norm=False, turn=0)
    one, two = c.cache(), c.cache()
    got = c.call(one, positions=None)
    B.kv_write(two, c.k.cuda(), c.v.cuda(), torch.from_numpy(c.slots).cuda())
    assert torch.equal(got.cpu(), c.q)
    assert all(torch.equal(one.tensors[i], two.tensors[i]) for i in (0, 1, 3, 4))


@pytest.mark.parametrize("rule", ["absmax", "sweep"])
def test_slots_and_positions_out_of_range(rule):
    """A slot that is none: nothing is written, q is there.  A position that is none: nothing is written, q is NaN."""
    c = Case(14, rule=rule, drop=((0, -1), (5, 0), (7, 1 << 40)), lost=((2, -1), (5, 0), (9, 1 << 40), (12, -(1 << 62))))
    c.check()
    q = c.expected()[0]
    assert torch.isnan(q[[2, 5, 9, 12]]).all() and torch.isfinite(q[[0, 7]]).all()
    empty = Case(15, rule=rule)
    empty.table = empty.table[:0]
    empty.reach = 0
    cache = empty.cache()
    assert torch.isnan(empty.call(cache)).all() and all((cache.tensors[i] == 0xA5).all() for i in (0, 1, 3, 4))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rule,dtype", [("absmax", BF16), ("absmax", F32), ("sweep", BF16)])
def test_one_buffer_of_q_k_v_in_place(rule, dtype, interleaved):
    """q, k and v as parts of one projection's rows, q turned in place; k and v stay."""
    c = Case(16, rule=rule, dtype=dtype, turn=96, interleaved=interleaved, tokens=301, reach=900)
    H, G, D = c.heads, c.group, c.dim
    both = torch.cat((c.q, c.k, c.v), 1).cuda()
    kept = both.clone()
    q, k, v = both[:, :H * G], both[:, H * G:H * G + H], both[:, H * G + H:]
    cache = c.cache()
    assert c.call(cache, q=q, k=k, v=v, out=q) is q
    want, sides, good = c.expected()
    assert same(q, want) and torch.equal(both[:, H * G:], kept[:, H * G:])
    c.check_cache(cache, sides, good)


def test_strides():
    """Heads outside tokens, tables and outputs with gaps."""
    c = Case(17, turn=64)
    def wide(x):
        w = torch.zeros(x.shape[1], x.shape[0] + 3, 2 * c.dim, dtype=x.dtype, device="cuda")
        w[:, :x.shape[0], c.dim:] = x.cuda().transpose(0, 1)
        return w[:, :x.shape[0], c.dim:].transpose(0, 1)
    table = torch.zeros(c.reach, 100, device="cuda")
    table[:, 4:68] = torch.from_numpy(c.table).cuda()
    hold = torch.full((c.tokens, 2, c.heads * c.group, c.dim), 7.0, dtype=BF16, device="cuda")
    cache = c.cache()
    got = c.call(cache, q=wide(c.q), k=wide(c.k), v=wide(c.v), rope=table[:, 4:68], out=hold[:, 1])
    want, sides, good = c.expected()
    assert same(got, want) and (hold[:, 0] == 7.0).all()
    c.check_cache(cache, sides, good)


@pytest.mark.parametrize("big", [1e30, 1e-30])
def test_norms_of_large_and_small_rows(big):
    """Squares that leave binary32 do not leave binary64."""
    c = Case(18, dtype=F32, turn=64)
    c.q, c.k, c.eps = c.q * big, c.k * big, 1e-12 if big > 1 else 1e-37
    c.check()


def test_empty():
    c = Case(19)
    cache = c.cache()
    out = B.kv_append(cache, c.k[:0].cuda(), c.v[:0].cuda(), torch.zeros(0, dtype=torch.int64, device="cuda"), q=c.q[:0].cuda())
    assert out.shape == (0, 6, 128) and all((cache.tensors[i] == 0xA5).all() for i in (0, 1, 3, 4))


def test_tables():
    """rope_table and rope_frequencies against binary64 numpy."""
    t = B.rope_table(1000, 64, base=500000.0, factor=4.0, magnitude=1.25).cpu().double().numpy()
    f = 500000.0 ** (-np.arange(32) / 32)
    a = np.arange(1000)[:, None] / 4.0 * f
    want = 1.25 * np.concatenate((np.cos(a), np.sin(a)), 1)
    # one rounding, and a few 2^-52 of angles up to 250 in the arguments
    assert np.abs(t - want).max() <= 1.25 * 2.0 ** -24 + 1e-12
    g = B.rope_frequencies(64, base=10000.0, factor=8.0, original_length=4096).cpu().numpy()
    f = 10000.0 ** (-np.arange(32) / 32)
    turns = 4096 * f / (2 * np.pi)
    assert np.allclose(g[turns > 40], f[turns > 40], rtol=1e-12) and np.allclose(g[turns < 0.8], f[turns < 0.8] / 8, rtol=1e-12)
    assert (g <= f * (1 + 1e-12)).all() and (g >= f / 8 * (1 - 1e-12)).all() and (np.diff(g) < 0).all()
    assert np.allclose(B.rope_frequencies(64, factor=8.0).cpu().numpy(), f / 8, rtol=1e-12)
    custom = B.rope_table(10, 64, frequencies=g).cpu().numpy()
    assert np.abs(custom[:, :32] - np.cos(np.arange(10)[:, None] * g)).max() < 1e-7


@pytest.mark.parametrize("rule", ["absmax", "sweep"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_a_row_with_infinities(dtype, rule):
    """1 / infinity is 0: the row's finite values become zeros, the infinite ones NaN; a NaN is the whole row's."""
    c = Case(20, rule=rule, dtype=dtype, turn=0)
    c.q[1, 2, 40], c.q[3, 0, 0], c.q[3, 0, 127], c.q[5, 4, 9] = float("inf"), float("inf"), -float("inf"), float("nan")
    want, sides, good = c.expected()
    assert (want[1, 2] == 0).sum() == 127 and torch.isnan(want[5, 4]).all()
    cache = c.cache()
    assert same(c.call(cache), want)
    c.check_cache(cache, sides, good)
