"""GPU parity of the calls around running requests: norms and rotation of
queries and keys with the row write, and forking, freeing, compacting and
copying the blocks of a paged cache, each against a plain implementation in 64
bits or in whole numbers.

Tolerance of the rotation.  Everything is fp32 until one rounding to bf16, off
by 2^-8 of the value at most.  Before it: a sum of D <= 256 squares, each product
and addition off by 2^-24 of the sum, is off by 257 2^-24 < 2^-15.9 of it, its
root by half as much, and the reciprocal root, three products and the sum of two
by less than 2^-20 of |a c| + |b s|.  So
|out - ref| <= 2^-8 |ref| + 2^-16 (|a c| + |b s|), rounded up to 2^-15.
"""
import math
import random

import numpy as np
import pytest
import torch

import grouped_query_kv_gb300 as g

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_query_kv_gb300 import build
    build.build()
    g.set_tuning(0, 0)
    yield


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, seed):
    return torch.randn(shape, generator=_gen(seed), device="cuda").to(torch.bfloat16)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _raises(status):
    with pytest.raises(g.KvAttnError) as ei:
        g.check_device_error()
    assert ei.value.status == status
    g.check_device_error()


# ------------------------------------------------------- norms and rotation

def rope_tables(max_pos, rd, base=10000.0):
    f = base ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float(), a.sin().float()


def rope_ref(x, w, pos, cos, sin, eps, interleaved):
    """(result, |a c| + |b s|) in 64 bits of rows with a position, zeros of the others."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    rd = 2 * cos.shape[1]
    ok = (pos >= 0) & (pos < cos.shape[0])
    at = torch.where(ok, pos, 0).long()
    c, s = cos.double()[at][:, None], sin.double()[at][:, None]
    first, second = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    a, b = x[..., first], x[..., second]
    y, mag = x.clone(), x.abs()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    mag[..., first], mag[..., second] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    return torch.where(ok[:, None, None], y, 0.0), torch.where(ok[:, None, None], mag, 0.0)


def check_rope(out, ref, mag):
    o = out.double()
    assert bool(torch.isfinite(o).all())
    over = (o - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -15 * mag)
    assert float(over.max()) <= 0, float(over.max())


def rope_inputs(N, Hq, Hkv, D, rd, max_pos, seed, pad=0, norm=True):
    qkv = _normal((N, Hq + 2 * Hkv, D), seed)
    pos = torch.randint(0, max_pos, (N,), generator=_gen(seed + 1), device="cuda", dtype=torch.int32)
    pos[0] = max_pos - 1
    if pad:
        pos[-pad:] = -1
        qkv[-pad:] = NAN
    w = [1 + 0.25 * torch.randn(D, generator=_gen(seed + 2 + i), device="cuda") if norm else None for i in range(2)]
    cos, sin = rope_tables(max_pos, rd)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, cos, sin, w[0], w[1]


SHAPES = [(64, 4, 1, 64), (64, 1, 1, 32), (64, 15, 3, 48), (128, 64, 8, 128), (128, 5, 1, 16), (128, 3, 3, 96),
          (256, 16, 1, 256), (256, 2, 2, 128), (256, 48, 1, 240)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,rd", SHAPES)
def test_rope(D, Hq, Hkv, rd, norm, interleaved):
    for N, pad in ((1, 0), (67, 5)):
        q, k, v, pos, cos, sin, qw, kw = rope_inputs(N, Hq, Hkv, D, rd, 1000, seed=D + Hq + N, pad=pad, norm=norm)
        qo, ko = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw, eps=1e-5, interleaved=interleaved)
        g.check_device_error()
        fine = (pos >= 0)[:, None, None]
        for x, w, out in ((q, qw, qo), (k, kw, ko)):
            ref, mag = rope_ref(torch.where(fine, x, 0.0), w, pos, cos, sin, 1e-5, interleaved)
            check_rope(out, ref, mag)
            if pad:
                assert not bool(out[-pad:].view(torch.int16).any())


@pytest.mark.parametrize("D,Hq,Hkv,bs", [(64, 6, 2, 16), (128, 64, 8, 64), (256, 3, 1, 32)])
def test_rope_rows_go_to_their_slots(D, Hq, Hkv, bs):
    N, pad, nblk = 83, 4, 9
    q, k, v, pos, cos, sin, qw, kw = rope_inputs(N, Hq, Hkv, D, D, 500, seed=D, pad=pad)
    slots = torch.randperm(nblk * bs, generator=_gen(3), device="cuda")[:N]
    slots[7] = -1  # a row that is not kept
    slots[11] = -5
    pools = [torch.full((nblk, Hkv, bs, D), 7.25, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qo = g.kv_append_rope(q, k, v, pos, cos, sin, slots, *pools, q_weight=qw, k_weight=kw, eps=1e-5)
    g.check_device_error()
    q2, k2 = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw, eps=1e-5)
    assert torch.equal(qo.view(torch.int16), q2.view(torch.int16))
    written = (slots >= 0) & (pos >= 0)
    want = [torch.full_like(p, 7.25) for p in pools]
    at = slots[written]
    for p, x in zip(want, (k2, v)):
        p[at // bs, :, at % bs] = x[written]
    for p, w in zip(pools, want):
        assert torch.equal(p.view(torch.int16), w.view(torch.int16))
    # one weight alone: the other side passes through the rotation only
    qo = g.kv_append_rope(q, k, v, pos, cos, sin, slots, *pools, k_weight=kw, eps=1e-5)
    ref, mag = rope_ref(torch.where((pos >= 0)[:, None, None], q, 0.0), None, pos, cos, sin, 1e-5, False)
    check_rope(qo, ref, mag)


def test_rope_in_place_and_into_wider_rows():
    q, k, v, pos, cos, sin, qw, kw = rope_inputs(50, 8, 2, 128, 64, 100, seed=9)
    q1, k1 = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw)
    wide = _normal((50, 16, 128), 4)
    before = wide.clone()
    g.qk_norm_rope(q, k, pos, cos, sin, qw, kw, q_out=wide[:, 3:11], k_out=wide[:, 13:15])
    assert torch.equal(wide[:, 3:11], q1) and torch.equal(wide[:, 13:15], k1)
    for a, e in ((0, 3), (11, 13), (15, 16)):
        assert torch.equal(wide[:, a:e], before[:, a:e])
    v0 = v.clone()
    out = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw, q_out=q, k_out=k)
    assert out[0] is q and torch.equal(q, q1) and torch.equal(k, k1) and torch.equal(v, v0)
    g.check_device_error()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 40, 4), (128, 64, 8), (256, 16, 1), (128, 1, 1)])
def test_rope_of_a_row_is_the_same_beside_any_others(D, Hq, Hkv):
    # (a call's heads are divided by the number of its tokens)
    q, k, v, pos, cos, sin, qw, kw = rope_inputs(2100, Hq, Hkv, D, D, 500, seed=D + 1)
    qa, ka = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw)
    for N in (1, 9, 64, 257, 600, 1100):
        qo, ko = g.qk_norm_rope(q[:N], k[:N], pos[:N], cos, sin, qw, kw)
        g.check_device_error()
        assert torch.equal(qo.view(torch.int16), qa[:N].view(torch.int16))
        assert torch.equal(ko.view(torch.int16), ka[:N].view(torch.int16))
        pools = [torch.zeros((N // 16 + 1, Hkv, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        mine = q[:N].clone(memory_format=torch.contiguous_format)
        back = g.kv_append_rope(mine, k[:N], v[:N], pos[:N], cos, sin, torch.arange(N, device="cuda"), *pools,
                                q_weight=qw, k_weight=kw, q_out=mine)
        g.check_device_error()
        assert back is mine and torch.equal(mine.view(torch.int16), qo.view(torch.int16))
        for p, x in zip(pools, (ka, v)):
            got = p.permute(0, 2, 1, 3).reshape(-1, Hkv, D)
            assert torch.equal(got[:N].view(torch.int16), x[:N].view(torch.int16)) and not bool(got[N:].any())


def test_rope_bad_positions_and_slots_are_reported():
    q, k, v, pos, cos, sin, qw, kw = rope_inputs(20, 4, 2, 64, 64, 30, seed=2)
    clean, _ = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw)
    bad = pos.clone()
    bad[5] = 30
    bad[6] = 2 ** 31 - 1
    bad[7] = -2 ** 31
    slots = torch.arange(20, device="cuda")
    pools = [torch.full((2, 2, 16, 64), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qo = g.kv_append_rope(q, k, v, bad, cos, sin, slots, *pools, q_weight=qw, k_weight=kw)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    rows = torch.tensor([i for i in range(20) if i not in (5, 6, 7)], device="cuda")
    assert torch.equal(qo[rows], clean[rows]) and not bool(qo[5:8].any())
    flat = pools[1].permute(0, 2, 1, 3).reshape(32, 2, 64)
    assert torch.equal(flat[rows], v[rows]) and bool((flat[5:8] == 3).all()) and bool((flat[20:] == 3).all())
    slots[3], slots[4] = 32, 2 ** 62
    kept = pools[0].clone()
    g.kv_append_rope(q, k, v, pos, cos, sin, slots, *pools)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    assert torch.equal(pools[0][0, :, 3:5], kept[0, :, 3:5])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_rows_that_hold_infinities_or_tiny_values(interleaved):
    q, k, v, pos, cos, sin, qw, kw = rope_inputs(6, 4, 2, 128, 64, 30, seed=5)
    q[1, 2, 100] = float("inf")  # not rotated: it stays where it is
    qo, _ = g.qk_norm_rope(q, k, pos, cos, sin, interleaved=interleaved)
    assert math.isinf(float(qo[1, 2, 100])) and bool(torch.isfinite(qo[1, 2, :100]).all())
    q[2] = 0
    q[3] *= 2.0 ** -60
    q[1, 2, 100] = 1
    qo, _ = g.qk_norm_rope(q, k, pos, cos, sin, qw, kw, eps=1e-6, interleaved=interleaved)
    ref, mag = rope_ref(q, qw, pos, cos, sin, 1e-6, interleaved)
    check_rope(qo, ref, mag)
    assert not bool(qo[2].any())


def test_rope_past_32_bits():
    # 300 000 rows of 64 heads of 128: 2.5e9 values of q
    N, Hq, Hkv, D = 300_000, 64, 1, 128
    q = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    for a in range(0, N, 50_000):
        q[a:a + 50_000] = _normal((50_000, Hq, D), a)
    k = _normal((N, Hkv, D), 1)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") % 4096
    cos, sin = rope_tables(4096, 128)
    qo, ko = g.qk_norm_rope(q, k, pos, cos, sin)
    g.check_device_error()
    for a in (0, 131_000, 262_140, N - 64):  # (rows about 2^31 values, and the last)
        ref, mag = rope_ref(q[a:a + 64], None, pos[a:a + 64], cos, sin, 0, False)
        check_rope(qo[a:a + 64], ref, mag)
    ref, mag = rope_ref(k, None, pos, cos, sin, 0, False)
    check_rope(ko, ref, mag)


# ------------------------------------------------------------------- blocks

class Pool:
    """The blocks of a paged cache in whole numbers, as the header describes them."""

    def __init__(self, R, maxb, nblk, bs, nfree=None):
        self.bs, self.maxb, self.nblk = bs, maxb, nblk
        self.table = np.full((R, maxb), -1, dtype=np.int64)
        self.lens = np.zeros(R, dtype=np.int64)
        self.refs = np.zeros(nblk, dtype=np.int64)
        self.free = list(range(nblk))
        self.size = nfree or nblk

    def blocks(self, n):
        return -(-int(n) // self.bs)

    def grow(self, r, n):
        for e in range(self.blocks(self.lens[r]), self.blocks(self.lens[r] + n)):
            self.table[r, e] = self.free.pop()
        self.lens[r] += n

    def fork(self, parents, children):
        copies = []
        for p, c in zip(parents, children):
            n = int(self.lens[p])
            self.lens[c] = n
            whole = n // self.bs
            self.table[c, :whole] = self.table[p, :whole]
            np.add.at(self.refs, self.table[p, :whole], 1)
            if n % self.bs:
                self.table[c, whole] = self.free.pop()
                copies.append((self.table[p, whole], self.table[c, whole]))
            else:
                copies.append((-1, -1))
        return np.array(copies).reshape(-1, 2)

    def drop(self, rows):
        gone = []
        for r in dict.fromkeys(rows):
            for e in range(self.blocks(self.lens[r])):
                b = self.table[r, e]
                self.refs[b] -= 1
                if self.refs[b] < 0:
                    gone.append(b)
                    self.refs[b] = 0
                self.table[r, e] = -1
            self.lens[r] = 0
        self.free += sorted(gone)

    def compact(self):
        free = set(self.free)
        used = self.nblk - len(free)
        remap = np.array([-1 if b in free else b for b in range(self.nblk)])
        holes = [b for b in range(used) if b in free]
        movers = [b for b in range(used, self.nblk) if b not in free]
        moves = np.full((self.nblk // 2, 2), -1)
        for i, (src, dst) in enumerate(zip(movers, holes)):
            moves[i] = src, dst
            remap[src] = dst
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for r in range(len(self.lens)):
            nb = self.blocks(self.lens[r])
            self.table[r, :nb] = remap[self.table[r, :nb]]
        self.free = list(range(self.nblk - 1, used - 1, -1))
        return moves, remap


class Device:
    """The same on the GPU."""

    def __init__(self, pool):
        self.bs = pool.bs
        self.table, self.lens, self.refs = (_i32(x) for x in (pool.table, pool.lens, pool.refs))
        self.free = torch.full((pool.size,), -1, dtype=torch.int32, device="cuda")
        self.free[:len(pool.free)] = _i32(pool.free)
        self.count = _i32([len(pool.free)])

    def args(self):
        return self.table, self.lens, self.refs, self.free, self.count

    def same(self, pool):
        assert int(self.count) == len(pool.free)
        for mine, theirs in ((self.table, pool.table), (self.lens, pool.lens), (self.refs, pool.refs),
                             (self.free[:len(pool.free)], pool.free)):
            assert np.array_equal(mine.cpu().numpy(), np.asarray(theirs).astype(np.int32))


@pytest.mark.parametrize("R,maxb,nblk,bs,most", [(1, 1, 3, 16, 1), (12, 5, 40, 16, 4), (40, 33, 900, 64, 20),
                                                 (600, 70, 20000, 16, 250), (3000, 12, 9001, 128, 1500)])
def test_forks_drops_and_compactions_in_turns(R, maxb, nblk, bs, most):
    rng = random.Random(R)
    pool = Pool(R, maxb, nblk, bs)
    rng.shuffle(pool.free)
    for r in range(0, R, 2):
        n = rng.choice([0, 1, bs, bs - 1, bs + 1, maxb * bs, rng.randint(0, maxb * bs)])
        n = min(n, maxb * bs)
        if pool.blocks(n) <= len(pool.free) // 2:
            pool.grow(r, n)
    dev = Device(pool)
    for turn in range(6):
        idle = [r for r in range(R) if pool.lens[r] == 0]
        busy = [r for r in range(R) if pool.lens[r] > 0]
        rng.shuffle(idle)
        k = min(len(idle), most, len(pool.free))
        if k and busy:
            parents, children = [rng.choice(busy) for _ in range(k)], idle[:k]  # (parents may come twice)
            copies, count = g.kv_fork_blocks(*dev.args(), _i32(parents), _i32(children), bs)
            g.check_device_error()
            assert np.array_equal(copies.cpu().numpy(), pool.fork(parents, children))
            assert count is dev.count
            dev.same(pool)
        busy = [r for r in range(R) if pool.lens[r] > 0]
        rows = [rng.choice(busy) for _ in range(max(1, len(busy) // 3))] if busy else []
        rows += rng.sample(range(R), min(R, 3))  # (some twice, some of length 0)
        g.kv_free_blocks(*dev.args(), _i32(rows), bs)
        g.check_device_error()
        pool.drop(rows)
        dev.same(pool)
        if turn % 2:
            before = [t.clone() for t in dev.args()]
            outs = [torch.zeros_like(t) for t in before]
            moves, remap = g.kv_compact_blocks(*dev.args(), bs, block_table_out=outs[0], refs_out=outs[2],
                                               free_blocks_out=outs[3], free_count_out=outs[4])
            g.check_device_error()
            for t, b in zip(dev.args(), before):
                assert torch.equal(t, b)
            m2, r2 = g.kv_compact_blocks(*dev.args(), bs)
            g.check_device_error()
            assert torch.equal(moves, m2) and torch.equal(remap, r2)
            for i in (0, 2, 3, 4):
                assert torch.equal(outs[i], dev.args()[i])
            want_moves, want_remap = pool.compact()
            assert np.array_equal(moves.cpu().numpy(), want_moves)
            assert np.array_equal(remap.cpu().numpy(), want_remap)
            dev.same(pool)
            # nothing is left to move
            m3, _ = g.kv_compact_blocks(*dev.args(), bs)
            assert bool((m3 == -1).all())
            dev.same(pool)


def test_a_fork_of_many_and_all_dropped():
    # the most that a call names: every block shared 65 534 times
    R, bs = 65535, 16
    pool = Pool(R, 2, 65600, bs)
    pool.grow(0, bs + 3)
    dev = Device(pool)
    children = list(range(1, R))
    copies, _ = g.kv_fork_blocks(*dev.args(), _i32([0] * len(children)), _i32(children), bs)
    g.check_device_error()
    assert np.array_equal(copies.cpu().numpy(), pool.fork([0] * len(children), children))
    dev.same(pool)
    rows = list(range(R))
    random.Random(1).shuffle(rows)
    g.kv_free_blocks(*dev.args(), _i32(rows), bs)
    g.check_device_error()
    pool.drop(rows)
    dev.same(pool)


def test_forks_that_cannot_be_served():
    bs = 16
    pool = Pool(10, 4, 12, bs)
    for r, n in ((0, 40), (1, 16), (2, 5)):
        pool.grow(r, n)
    pool.free = pool.free[:2]  # two blocks left
    dev = Device(pool)
    dev.lens[9] = 65  # longer than its row
    #         served, its child again, own row, a child's row, in use, outside, outside, too long, last block, none left
    parents = [0, 0, 3, 5, 0, 0, 10, 9, 2, 2, 1]
    children = [5, 5, 3, 6, 1, -1, 6, 6, 7, 8, 6]
    copies, _ = g.kv_fork_blocks(*dev.args(), _i32(parents), _i32(children), bs)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    want = np.full((11, 2), -1)
    served = [0, 8, 10]  # (the last needs no block, and comes after one that found none)
    # row 6 is marked first by fork 3, whose parent is a child: fork 10 does not get it
    served.remove(10)
    for i in served:
        want[i] = pool.fork([parents[i]], [children[i]])[0]
    assert np.array_equal(copies.cpu().numpy(), want)
    dev.lens[9] = 0
    dev.same(pool)


def test_bad_blocks_are_reported_and_the_others_served():
    bs = 16
    pool = Pool(6, 3, 20, bs)
    for r in range(3):
        pool.grow(r, 40)
    dev = Device(pool)
    dev.table[0, 1] = 20
    dev.table[1, 2] = -7
    copies, _ = g.kv_fork_blocks(*dev.args(), _i32([0, 1, 2]), _i32([3, 4, 5]), bs)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    t = dev.table.cpu().numpy()
    assert t[3, 1] == 20 and t[3, 0] == t[0, 0] and list(copies[1].cpu()) == [-1, -1]
    assert list(copies[2].cpu()) == [t[2, 2], t[5, 2]]
    refs = dev.refs.cpu().numpy()
    assert refs[t[0, 0]] == 1 and refs[t[2, 1]] == 1 and refs.sum() == 5
    count = int(dev.count)
    g.kv_free_blocks(*dev.args(), _i32([0, 3, 6, -1, 1]), bs)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    # of 0 and 3: the shared first block, both last ones; of 1: two, whose fork still holds them
    assert int(dev.count) == count + 3 and dev.lens.tolist() == [0, 0, 40, 0, 40, 40]
    assert sorted(dev.free[count:count + 3].tolist()) == dev.free[count:count + 3].tolist()
    # a count that is none: nothing happens
    before = [x.clone() for x in dev.args()]
    for bad in (-1, 21):
        dev.count.fill_(bad)
        g.kv_free_blocks(*dev.args(), _i32([2]), bs)
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        moves, remap = g.kv_compact_blocks(*dev.args(), bs)
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        assert bool((moves == -1).all()) and int(dev.count) == bad
        for x, b in list(zip(dev.args(), before))[1:4]:
            assert torch.equal(x, b)
    # more than the stack holds
    small = Device(pool)
    small.free = small.free[:int(small.count) + 1].clone()
    g.kv_free_blocks(*small.args(), _i32([2]), bs)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    assert int(small.count) == small.free.shape[0]


def test_compaction_of_stacks_and_tables_that_lie():
    bs = 16
    pool = Pool(2, 3, 9, bs)
    pool.free = [0, 1, 2, 3, 4, 5]
    pool.table[0, :2] = [8, 7]
    pool.table[1, :1] = [6]
    pool.lens[:] = [20, 3]
    dev = Device(pool)
    dev.free[:7] = _i32([5, 5, 0, 1, 44, 3, -2])  # 2 and 4 are missing: held by nobody known
    dev.count.fill_(7)
    dev.table[1, 0] = 3  # a free block
    moves, remap = g.kv_compact_blocks(*dev.args(), bs)
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    # held: 2, 4, 6, 7, 8 -> used = 5; holes 0, 1, 3
    assert remap.tolist() == [-1, -1, 2, -1, 4, -1, 0, 1, 3]
    assert moves.tolist() == [[6, 0], [7, 1], [8, 3], [-1, -1]]
    assert dev.table.tolist() == [[3, 1, -1], [-1, -1, -1]]
    assert int(dev.count) == 4 and dev.free[:4].tolist() == [8, 7, 6, 5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("Hkv,bs,D", [(1, 16, 64), (3, 16, 128), (8, 64, 128), (2, 1024, 256)])
def test_copy_blocks(Hkv, bs, D, dtype):
    nblk, n = 23, 9
    raw = [torch.randint(0, 256, (nblk, Hkv, bs, D * (2 if dtype is torch.bfloat16 else 1)), generator=_gen(i),
                         device="cuda", dtype=torch.uint8) for i in range(2)]
    pools = [r.view(dtype) for r in raw]
    ids = torch.randperm(nblk, generator=_gen(5), device="cuda", dtype=torch.int32)
    copies = torch.stack([ids[:n], ids[n:2 * n]], 1).contiguous()
    copies[0, 0] = copies[1, 0]  # one block to two places
    copies[4] = -1
    want = [r.clone() for r in raw]
    scales = want_s = None
    if dtype is torch.uint8:
        scales = [torch.rand((nblk, Hkv), generator=_gen(7 + i), device="cuda") for i in range(2)]
        want_s = [s.clone() for s in scales]
    for src, dst in copies.tolist():
        if src >= 0:
            for i in range(2):
                want[i][dst] = raw[i][src]
                if scales:
                    want_s[i][dst] = scales[i][src]
    g.kv_copy_blocks(*pools, copies, *(scales or ()))
    g.check_device_error()
    for i in range(2):
        assert torch.equal(raw[i], want[i])
        assert scales is None or torch.equal(scales[i], want_s[i])
    bad = _i32([[0, nblk], [-1, 3], [nblk, 1], [-2, -1], [2 ** 31 - 1, 0]])
    g.kv_copy_blocks(*pools, bad, *(scales or ()))
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    for i in range(2):
        assert torch.equal(raw[i], want[i])


def test_copy_blocks_past_32_bits():
    # pools of 5 GB each: a block at each end
    nblk, Hkv, bs, D = 5 * 2 ** 30 // (8 * 64 * 128 * 2), 8, 64, 128
    pools = [torch.zeros((nblk, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    a = _normal((2, Hkv, bs, D), 1)
    pools[0][0], pools[1][nblk - 2] = a[0], a[1]
    pools[1][0], pools[0][nblk - 2] = a[1], a[0]
    g.kv_copy_blocks(*pools, _i32([[0, nblk - 1], [nblk - 2, 1]]))
    g.check_device_error()
    for i in range(2):
        assert torch.equal(pools[i][nblk - 1], a[i]) and torch.equal(pools[i][1], a[i])
        assert not bool(pools[i][2:nblk - 2].any())


def test_few_rows_of_many_blocks_and_many_rows_of_few():
    for R, maxb, nblk, bs in ((4, 9000, 30000, 16), (1500, 3, 50000, 16), (300, 40, 33000, 32)):
        pool = Pool(R, maxb, nblk, bs)
        random.Random(R).shuffle(pool.free)
        for r in range(0, R, 2):
            pool.grow(r, maxb * bs - r % 5)
        dev = Device(pool)
        parents, children = list(range(0, R, 2))[:R // 2], list(range(1, R, 2))
        copies, _ = g.kv_fork_blocks(*dev.args(), _i32(parents), _i32(children), bs)
        g.check_device_error()
        assert np.array_equal(copies.cpu().numpy(), pool.fork(parents, children))
        dev.same(pool)
        rows = parents[::2] + children[1::2]
        g.kv_free_blocks(*dev.args(), _i32(rows), bs)
        g.check_device_error()
        pool.drop(rows)
        dev.same(pool)
        moves, remap = g.kv_compact_blocks(*dev.args(), bs)
        g.check_device_error()
        want_moves, want_remap = pool.compact()
        assert np.array_equal(moves.cpu().numpy(), want_moves) and np.array_equal(remap.cpu().numpy(), want_remap)
        dev.same(pool)


def test_a_request_s_life_forked_copied_compacted_and_dropped():
    # blocks, rows, attention; a fork that goes its own way; compaction; the drop
    Hq, Hkv, D, bs, R, nblk = 8, 2, 128, 16, 4, 24
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.full((R, 8), -1, **i32), torch.zeros(R, **i32)
    refs, free = torch.zeros(nblk, **i32), torch.arange(nblk - 1, -1, -1, **i32)
    free[[3, 20]] = free[[20, 3]]
    count = torch.tensor([nblk], **i32)
    pools = [torch.full((nblk, Hkv, bs, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cos, sin = rope_tables(200, D)
    hist = {r: [torch.zeros((0, Hkv, D), dtype=torch.float64, device="cuda")] * 2 for r in range(R)}

    def step(new, seed):
        n = sum(new)
        cu, slots, _ = g.kv_block_tables(lens, _i32(new), table, free, count, bs, n)
        qkv = _normal((n, Hq + 2 * Hkv, D), seed)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.cat([torch.arange(m, **i32) + lens[r] for r, m in enumerate(new)])
        qo = g.kv_append_rope(q, k, v, pos, cos, sin, slots, *pools)
        _, ko = g.qk_norm_rope(q, k, pos, cos, sin)
        lens.add_(_i32(new))
        out = g.gqa_extend_attn(qo, *pools, table, lens, cu, 0.1)
        g.check_device_error()
        at = 0
        for r, m in enumerate(new):
            if not m:
                continue
            hist[r] = [torch.cat([h, x[at:at + m].double()]) for h, x in zip(hist[r], (ko, v))]
            K, V = (h.repeat_interleave(Hq // Hkv, 1) for h in hist[r])
            e = K.shape[0]
            s = torch.einsum("ihd,jhd->hij", qo[at:at + m].double(), K) * 0.1
            s = s.masked_fill(torch.arange(e, device="cuda")[None, :] > torch.arange(e - m, e, device="cuda")[:, None],
                              -math.inf)
            w = torch.softmax(s, 2)
            ref, mag = torch.einsum("hij,jhd->ihd", w, V), torch.einsum("hij,jhd->ihd", w, V.abs())
            o = out[at:at + m].double()
            assert float(((o - ref).abs() - (2.0 ** -8 + 2.0 ** -10) * mag - 2.0 ** -8 * o.abs()).max()) <= 0
            at += m

    step([37, 20, 0, 0], 1)
    copies, _ = g.kv_fork_blocks(table, lens, refs, free, count, _i32([0, 1]), _i32([2, 3]), bs)
    g.kv_copy_blocks(*pools, copies)
    for a, b in ((0, 2), (1, 3)):
        hist[b] = list(hist[a])
    step([1, 13, 30, 1], 2)
    step([1, 1, 1, 1], 3)
    g.kv_free_blocks(table, lens, refs, free, count, _i32([0]), bs)  # its fork keeps the shared blocks
    hist[0] = [h[:0] for h in hist[0]]
    moves, _ = g.kv_compact_blocks(table, lens, refs, free, count, bs)
    g.kv_copy_blocks(*pools, moves)
    used = nblk - int(count)
    assert int(table.max()) < used
    for p in pools:  # nothing is read from behind the used blocks
        p[used:] = NAN
    step([0, 1, 20, 2], 4)
    step([5, 1, 1, 1], 5)
    g.kv_free_blocks(table, lens, refs, free, count, _i32([0, 1, 2, 3]), bs)
    g.check_device_error()
    assert int(count) == nblk and not bool(refs.any()) and sorted(free.tolist()) == list(range(nblk))


def test_on_another_stream_and_captured():
    Hq, Hkv, D, bs = 8, 2, 128, 16
    q, k, v, pos, cos, sin, qw, kw = rope_inputs(64, Hq, Hkv, D, D, 500, seed=3)
    slots = torch.randperm(128, generator=_gen(1), device="cuda")[:64]
    pool = Pool(40, 6, 200, bs)
    for r in range(20):
        pool.grow(r, 5 + 4 * r)
    dev = Device(pool)
    start = [t.clone() for t in dev.args()]
    parents, children = _i32(range(20)), _i32(range(20, 40))
    pools = [_normal((200, Hkv, bs, D), 9 + i) for i in range(2)]
    first = [p.clone() for p in pools]
    copies = torch.zeros((20, 2), dtype=torch.int32, device="cuda")
    qo, moves, remap = torch.zeros_like(q, memory_format=torch.contiguous_format), None, None
    moves, remap = torch.zeros((100, 2), dtype=torch.int32, device="cuda"), torch.zeros(200, dtype=torch.int32, device="cuda")

    def path(**more):
        g.kv_append_rope(q, k, v, pos, cos, sin, slots, *pools, q_weight=qw, k_weight=kw, q_out=qo, **more)
        g.kv_fork_blocks(*dev.args(), parents, children, bs, copies=copies, **more)
        g.kv_copy_blocks(*pools, copies, **more)
        g.kv_free_blocks(*dev.args(), parents, bs, **more)
        g.kv_compact_blocks(*dev.args(), bs, moves=moves, remap=remap, **more)
        g.kv_copy_blocks(*pools, moves, **more)

    def reset():
        for t, s in zip(dev.args(), start):
            t.copy_(s)
        for p, f in zip(pools, first):
            p.copy_(f)
        qo.zero_()

    def state():
        torch.cuda.synchronize()
        g.check_device_error()
        return [t.clone() for t in (*dev.args(), *pools, qo, copies, moves, remap)]

    path()
    want = state()
    pool.fork(range(20), range(20, 40))
    pool.drop(range(20))
    pool.compact()
    dev.same(pool)
    side = torch.cuda.Stream()
    reset()
    torch.cuda.synchronize()
    busy = torch.cuda._sleep  # the current stream is busy meanwhile
    busy(20_000_000)
    path(stream=side)
    for a, b in zip(state(), want):
        assert torch.equal(a, b)
    reset()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        path()
    for _ in range(3):
        reset()
        gr.replay()
        for a, b in zip(state(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("aside", [False, True])
def test_empty_lists_and_a_pool_of_one_block(aside):
    bs, Hkv, D = 16, 2, 64
    pool = Pool(3, 4, 6, bs)
    pool.grow(0, 40)
    dev = Device(pool)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    more = dict(stream=torch.cuda.Stream()) if aside else {}
    torch.cuda.synchronize()
    # forks and drops of nobody: the count is passed on, all else stays
    copies, count = g.kv_fork_blocks(*dev.args(), none, none, bs, **more)
    assert copies.shape == (0, 2) and count is dev.count
    assert g.kv_free_blocks(*dev.args(), none, bs, **more) is dev.count
    for call in (lambda o: g.kv_fork_blocks(*dev.args(), none, none, bs, free_count_out=o, **more)[1],
                 lambda o: g.kv_free_blocks(*dev.args(), none, bs, free_count_out=o, **more)):
        out = _i32([-7])
        torch.cuda.synchronize()
        assert call(out) is out
        torch.cuda.synchronize()
        assert int(out) == 3
    # their checks stay
    with pytest.raises(ValueError):
        g.kv_fork_blocks(*dev.args(), none, _i32([1]), bs)
    with pytest.raises(TypeError):
        g.kv_free_blocks(*dev.args(), none.long(), bs)
    for dtype in (torch.bfloat16, torch.uint8):
        pools = [torch.full((6, Hkv, bs, D), 3, dtype=dtype, device="cuda") for _ in range(2)]
        scales = {}
        if dtype is torch.uint8:
            scales = {k: torch.ones(6, Hkv, device="cuda") for k in ("k_scale", "v_scale")}
        torch.cuda.synchronize()
        g.kv_copy_blocks(*pools, copies, **scales, **more)
        with pytest.raises(ValueError):
            g.kv_copy_blocks(pools[0], pools[1][:5], copies, **scales)
        torch.cuda.synchronize()
        assert all(bool((p == 3).all()) for p in pools)
    g.check_device_error()
    dev.same(pool)
    # a pool of one block, free or held
    for n in (0, 9):
        one = Pool(1, 1, 1, bs)
        one.grow(0, n)
        dev = Device(one)
        pools = [torch.ones((1, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        moves, remap = g.kv_compact_blocks(*dev.args(), bs, **more)
        assert moves.shape == (0, 2)
        g.kv_copy_blocks(*pools, moves, **more)
        torch.cuda.synchronize()
        g.check_device_error()
        assert remap.tolist() == [0 if n else -1]
        dev.same(one)
