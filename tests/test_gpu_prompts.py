"""GPU parity of the calls that take prompts into a paged cache: block tables
and slot maps, packed row writes, prompt attention, and the 8-bit pool with a
scale per block and K/V head, each against a plain implementation in 64 bits.

Tolerances.  A rounding is off by at most half a step: 2^-8 for bf16, 2^-11
for binary16, relative to the value.
 * Prompt attention: the weights are rounded to bf16 (2^-8 of each) and the
   result once more (2^-8 of it).  A score of D products in fp32 is off by at
   most D 2^-24 sum|q k| scale, which moves a weight and the weights' sum by as
   much, relatively: with N(0,1) inputs sum|q k| scale <= 0.7 sqrt(D) + a few,
   under 2^-11 together at D = 256.  So |out - ref| <= (2^-8 + 2^-10)
   sum_j w_j |v_j| + 2^-8 |out|.
 * Attention over the 8-bit pool: see attn8_bound.
"""
import math

import numpy as np
import pytest
import torch

import grouped_query_kv_gb300 as g
from helpers import bits

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_query_kv_gb300 import build
    build.build()
    g.set_tuning(0, 0)
    g.set_wait_limit(0)
    yield
    g.set_wait_limit(0)
    g.set_tuning(0, 0)


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


# ------------------------------------------------------------ prompt attention

def prefill_ref(q, k, v, cu, scale, window=None):
    """(out, sum of weights times |v|) in 64 bits; NaN in rows of no sequence."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.full((N, Hq, D), NAN, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    for a, e in zip(cu[:-1], cu[1:]):
        if e <= a:
            continue
        qs = q[a:e].double().permute(1, 0, 2)
        ks = k[a:e].double().permute(1, 0, 2).repeat_interleave(G, 0)
        vs = v[a:e].double().permute(1, 0, 2).repeat_interleave(G, 0)
        s = qs @ ks.transpose(1, 2) * scale
        i = torch.arange(e - a, device=q.device)
        far = i[:, None] - i[None, :]
        s[:, (far < 0) | (far >= (window or e - a))] = -math.inf
        w = torch.softmax(s, dim=2)
        out[a:e] = (w @ vs).permute(1, 0, 2)
        mag[a:e] = (w @ vs.abs()).permute(1, 0, 2)
    return out, mag


def check_prefill(out, ref, mag, before=None):
    mine = ~torch.isnan(ref[:, 0, 0])
    o = out.double()
    assert bool(torch.isfinite(o[mine]).all())
    over = (o - ref)[mine].abs() - ((2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * o.abs())[mine]
    assert float(over.max()) <= 0 if over.numel() else True, float(over.max())
    if before is not None:  # rows of no sequence: bit for bit what they were
        assert torch.equal(out[~mine].view(torch.int16), before[~mine].view(torch.int16))


def run_prefill(lens, Hq, Hkv, D, seed, window=None, gaps=0, wide=True, scale=None, pad=3):
    starts = [gaps]
    for n in lens:
        starts.append(starts[-1] + n)
    N = starts[-1] + pad
    if wide:
        qkv = _normal((N, Hq + 2 * Hkv, D), seed)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (_normal((N, h, D), seed + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    for t in (q, k, v):  # rows of no sequence hold NaN
        t[:gaps] = NAN
        t[starts[-1]:] = NAN
    before = torch.full((N, Hq, D), 7.25, dtype=torch.bfloat16, device="cuda")
    out = before.clone()
    scale = 1 / math.sqrt(D) if scale is None else scale
    g.gqa_prefill_attn(q, k, v, _i32(starts), scale, out=out, window=window)
    g.check_device_error()
    ref, mag = prefill_ref(q, k, v, starts, scale, window)
    check_prefill(out, ref, mag, before)
    return out


HEADS = [(64, 4, 1), (64, 6, 2), (64, 3, 3), (128, 64, 8), (128, 8, 8), (128, 5, 1), (128, 32, 1),
         (256, 16, 1), (256, 48, 1), (256, 3, 1), (256, 4, 4), (128, 256, 1)]


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_prefill_one_token(D, Hq, Hkv):
    run_prefill([1], Hq, Hkv, D, seed=1, pad=0)


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_prefill_lengths_at_tile_edges(D, Hq, Hkv):
    run_prefill([0, 1, 2, 15, 16, 17, 0, 31, 33, 63, 64, 65, 127, 128, 129, 143, 144, 255, 256, 257, 300, 1], Hq,
                Hkv, D, seed=D + Hq)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 1), (128, 64, 8), (128, 3, 3), (256, 16, 1), (256, 2, 2)])
@pytest.mark.parametrize("ctas", [0, 1, 5])
def test_prefill_long_prompts_and_small_grids(D, Hq, Hkv, ctas):
    g.set_tuning(0, ctas)
    try:
        run_prefill([1029, 3, 700, 0, 2065], Hq, Hkv, D, seed=3 * D + Hq, gaps=5)
    finally:
        g.set_tuning(0, 0)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 16, 2), (256, 16, 1), (256, 1, 1)])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 500, 4096])
def test_prefill_windows(D, Hq, Hkv, window):
    run_prefill([1, 130, 0, 777, 256, 1300], Hq, Hkv, D, seed=window + D, window=window, wide=False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 1.5])
def test_prefill_scales(D, scale):
    run_prefill([200, 77], 8, 2, D, seed=D, scale=scale)


def test_prefill_large_scores_move_the_running_max():
    # keys grow along the prompt, so later tiles raise the maximum by far more than 2^8
    D, Hq, Hkv, n = 128, 8, 2, 900
    for D in (64, 128, 256):
        q, k, v = _normal((n, Hq, D), 5), _normal((n, Hkv, D), 6), _normal((n, Hkv, D), 7)
        q = q.abs()
        k = (k.abs() * torch.linspace(0, 4, n, device="cuda")[:, None, None]).to(torch.bfloat16)
        cu = [0, n]
        out = g.gqa_prefill_attn(q, k, v, _i32(cu), 0.5)
        g.check_device_error()
        ref, mag = prefill_ref(q, k, v, cu, 0.5)
        # scores up to 0.5 * 4 * D * 0.64 <= 330: fp32 products and sums move a weight by
        # at most 2 (D + 2) 2^-24 330 <= 2^-6.6 at D = 256, so the weights' term is 2^-6.5 + 2^-8
        o = out.double()
        assert float(((o - ref).abs() - (2.0 ** -6.5 + 2.0 ** -8) * mag - 2.0 ** -8 * o.abs()).max()) <= 0


def test_prefill_many_sequences_and_one_long():
    # more than 256 blocks of one sequence (buckets of several blocks) among hundreds of short ones
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 5, 700).tolist()
    lens[123] = 4700
    run_prefill(lens, 16, 1, 128, seed=9)
    run_prefill(rng.integers(0, 3, 3000).tolist(), 4, 2, 64, seed=10)
    run_prefill([2500] + rng.integers(0, 40, 90).tolist(), 16, 1, 256, seed=11)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 4), (128, 16, 2), (256, 16, 1)])
def test_prefill_ragged_launches_back_to_back(D, Hq, Hkv):
    # many units of every number of key tiles in a CTA's list, three batches in
    # flight one behind the other: the copy ring turns over across all of them
    rng = np.random.default_rng(D)
    runs = []
    for i in range(3):
        lens = rng.permutation([0, 1, 130, 257, 700, 1400, 2049, 2900])
        cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
        q, k, v = (_normal((cu[-1], h, D), 7 * i + j) for j, h in enumerate((Hq, Hkv, Hkv)))
        runs.append((q, k, v, cu, _i32(cu)))
    for _ in range(3):
        outs = [g.gqa_prefill_attn(q, k, v, dcu, D ** -0.5) for q, k, v, _, dcu in runs]
    g.check_device_error()
    for (q, k, v, cu, _), out in zip(runs, outs):
        check_prefill(out, *prefill_ref(q, k, v, cu, D ** -0.5))


def test_prefill_neighbours_do_not_meet():
    # a sequence of NaN and infinities between two others: they come out as without it
    for D, Hq, Hkv in ((64, 4, 1), (128, 16, 2), (256, 4, 1)):
        lens = [45, 70, 51]
        q, k, v = (_normal((166, h, D), 20 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        cu = [0, 45, 115, 166]
        clean = g.gqa_prefill_attn(q, k, v, _i32(cu), 0.1)
        for t in (q, k, v):
            t[45:80] = NAN
            t[80:115] = math.inf
        out = g.gqa_prefill_attn(q, k, v, _i32(cu), 0.1)
        g.check_device_error()
        assert torch.equal(out[:45].view(torch.int16), clean[:45].view(torch.int16)), (D, lens)
        assert torch.equal(out[115:].view(torch.int16), clean[115:].view(torch.int16))


def test_prefill_flags_bad_bounds_and_serves_the_others():
    D, Hq, Hkv, N = 128, 8, 2, 120
    q, k, v = (_normal((N, h, D), 30 + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    for cu in ([0, 40, 30, 90], [-5, 20, 60, 100], [0, 50, 100, 121], [0, 50, 2 ** 31 - 1, 60]):
        out = torch.full((N, Hq, D), 2.0, dtype=torch.bfloat16, device="cuda")
        g.gqa_prefill_attn(q, k, v, _i32(cu), 0.1, out=out)
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        good = [(a, e) for a, e in zip(cu[:-1], cu[1:]) if 0 <= a <= e <= N]
        alone = (sum(((torch.arange(N) >= a) & (torch.arange(N) < e)).int() for a, e in good) == 1).cuda()
        for a, e in good:  # (rows of two sequences hold what either wrote)
            ref, mag = prefill_ref(q[a:e], k[a:e], v[a:e], [0, e - a], 0.1)
            ref[~alone[a:e]] = NAN
            check_prefill(out[a:e], ref, mag)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_a_wait_that_runs_out_reports_and_the_next_call_is_clean(D):
    g.check_device_error()
    q, k, v = _normal((600, 8, D), 1), _normal((600, 2, D), 2), _normal((600, 2, D), 3)
    cu = [0, 500, 600]
    try:
        g.set_wait_limit(1)
        g.gqa_prefill_attn(q, k, v, _i32(cu), 0.1)
        _raises(g.KVATTN_ERR_TIMEOUT)
    finally:
        g.set_wait_limit(0)
    out = g.gqa_prefill_attn(q, k, v, _i32(cu), 0.1)
    g.check_device_error()
    check_prefill(out, *prefill_ref(q, k, v, cu, 0.1))


def test_prefill_captured_replayed_and_on_two_streams():
    D, Hq, Hkv, N = 128, 16, 2, 700
    ts = [tuple(_normal((N, h, D), 40 + 3 * s + i) for i, h in enumerate((Hq, Hkv, Hkv))) for s in range(2)]
    cus = [[0, 300, 700], [0, 1, 690]]
    outs = [torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in ts]
    dev_cu = [_i32(c) for c in cus]
    graphs = []
    for t, cu, out in zip(ts, dev_cu, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):  # the first call, captured: nothing is allocated
            g.gqa_prefill_attn(*t, cu, 0.1, out=out)
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    g.check_device_error()
    for t, cu, out in zip(ts, cus, outs):
        ref, mag = prefill_ref(*t, cu, 0.1)
        check_prefill(out, ref, mag)
    dev_cu[0].copy_(_i32([0, 650, 651]))  # other lengths, the same graph
    graphs[0].replay()
    torch.cuda.synchronize()
    check_prefill(outs[0][:651], *(x[:651] for x in prefill_ref(*ts[0], [0, 650, 651], 0.1)))


def test_prefill_past_32_bits():
    # the last rows of a projection of 2^32 elements and more, out as well
    N, Hq, Hkv, D = 530000, 64, 8, 128
    qkv = torch.zeros((N, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    qkv[N - 300:] = _normal((300, Hq + 2 * Hkv, D), 1)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out = g.gqa_prefill_attn(q, k, v, _i32([N - 300, N - 170, N]), 0.1)
    g.check_device_error()
    last = [t[N - 300:].contiguous() for t in (q, k, v)]
    check_prefill(out[N - 300:], *prefill_ref(*last, [0, 130, 300], 0.1))
    assert not bool(out[:1000].any()) and not bool(out[N - 1000:N - 300].any())
    del qkv, q, k, v, out
    torch.cuda.empty_cache()


# ------------------------------------------------------------ tables and slots

def tables_ref(cached, new, table, free, count, bs, num_slots):
    """The rule of kv_block_tables; True if it flags an error."""
    table = table.copy()
    maxb = table.shape[1]
    bad = not 0 <= count <= len(free)
    if bad:
        count = 0
    cu, slots, taken, wanted = [0], [], 0, 0
    for b, (c, n) in enumerate(zip(cached, new)):
        ok = c >= 0 and n >= 0 and c + n <= maxb * bs
        rows = max(n, 0)
        cu.append(min(cu[-1] + rows, 2 ** 31 - 1))
        if not ok:
            bad = True
            slots += [-1] * min(rows, num_slots + 1)
            continue
        have, upto = -(-c // bs), -(-(c + n) // bs)
        wanted += upto - have
        if cu[-1] > num_slots or (upto > have and wanted > count):
            bad = True
            for e in range(have, upto):  # entries of rows that the slot map holds
                if cu[b] + e * bs - c < num_slots:
                    table[b, e] = -1
            slots += [-1] * rows
            continue
        for e in range(have, upto):
            taken += 1
            table[b, e] = free[count - taken]
        for p in range(c, c + n):
            blk = int(table[b, p // bs])
            slots.append(-1 if blk < 0 else blk * bs + p % bs)
    if len(slots) > num_slots:
        bad = True
    slots = (slots + [-1] * num_slots)[:num_slots]
    return table, np.array(cu), np.array(slots), count - taken, bad


def run_tables(cached, new, bs, maxb, num_free, count, num_slots=None, seed=0, in_place=True):
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached), np.asarray(new)
    table = np.full((len(cached), maxb), -1, np.int32)
    ids = rng.permutation(len(cached) * maxb + num_free).astype(np.int32)
    at = 0
    for b, c in enumerate(cached):
        n = min(max(-(-int(c) // bs), 0), maxb)
        table[b, :n] = ids[at:at + n]
        at += n
    free = ids[at:at + num_free]
    if num_slots is None:
        num_slots = max(1, int(np.maximum(new, 0).sum()) + 5)
    ref = tables_ref(cached.tolist(), new.tolist(), table, free.tolist(), count, bs, num_slots)
    d_table, d_count = _i32(table), _i32([count])
    slots = torch.full((num_slots,), 12345, dtype=torch.int64, device="cuda")
    left = None if in_place else torch.full((1,), 77, dtype=torch.int32, device="cuda")
    cu, slots, left = g.kv_block_tables(_i32(cached), _i32(new), d_table, _i32(free), d_count, bs, num_slots,
                                        slots=slots, free_count_out=left)
    if ref[4]:
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    else:
        g.check_device_error()
    assert np.array_equal(d_table.cpu().numpy(), ref[0])
    assert np.array_equal(cu.cpu().numpy(), ref[1])
    assert np.array_equal(slots.cpu().numpy(), ref[2])
    assert int(left) == ref[3]
    assert int(d_count) == (ref[3] if in_place else count)
    return ref


@pytest.mark.parametrize("B,bs,cmax,nmax", [(1, 16, 0, 1), (1, 16, 500, 1), (3, 16, 40, 1), (64, 16, 500, 1),
                                            (7, 32, 100, 300), (300, 16, 60, 90), (1024, 16, 33, 7),
                                            (1025, 16, 33, 7), (5000, 64, 200, 12), (2, 4096, 9000, 30000)])
def test_block_tables(B, bs, cmax, nmax):
    rng = np.random.default_rng(B + bs)
    for seed in range(3):
        cached, new = rng.integers(0, cmax + 1, B), rng.integers(0, nmax + 1, B)
        maxb = -(-(cmax + nmax) // bs) + 1
        need = int((-(-(cached + new) // bs) - -(-cached // bs)).sum())
        run_tables(cached, new, bs, maxb, need + 3, need + 3 - seed, seed=seed, in_place=seed != 1)


def test_block_tables_when_the_free_list_runs_out():
    for B, nmax in ((6, 50), (1500, 40)):
        rng = np.random.default_rng(B)
        cached, new = rng.integers(0, 60, B), rng.integers(0, nmax, B)
        new[::5] = 0
        need = int((-(-(cached + new) // 16) - -(-cached // 16)).sum())
        for count in (0, 1, need // 2, need - 1, need):
            run_tables(cached, new, 16, 8, need, count, seed=count)


def test_block_tables_bad_requests():
    run_tables([5, -1, 20, 3, 128], [3, 4, -7, 130, 1], 16, 8, 40, 40)     # negative or too long
    run_tables([5, 2 ** 31 - 1, 4], [3, 2 ** 31 - 1, 2], 16, 8, 9, 9, num_slots=30)
    run_tables([5, 7], [30, 40], 16, 8, 9, 9, num_slots=33)               # too few slots
    run_tables([5, 7], [30, 40], 16, 8, 9, -2)
    run_tables([5, 7], [30, 40], 16, 8, 9, 10)
    run_tables([3000, 7], [3000, 4000], 16, 600, 700, 700, num_slots=5000)  # the same with a large map


def test_block_tables_row_counts_that_add_up_past_32_bits():
    big = 2 ** 31 - 1
    run_tables([5, 7], [3, big], 16, 8, 9, 9, num_slots=30)          # behind other rows, last
    run_tables([5, 7, 1, 2], [29, big, big, 4], 16, 8, 9, 9, num_slots=30)
    run_tables([5, 7], [5000, big], 16, 400, 400, 400, num_slots=9001)  # from the second tile on
    run_tables([0] * 1500, [2] * 1499 + [big], 16, 8, 1500, 1500, num_slots=3001)


def test_append_slots_moves_bits():
    for D, Hkv, bs, N in ((64, 1, 16, 1), (64, 3, 32, 77), (128, 8, 16, 500), (256, 1, 128, 300), (256, 8, 16, 33)):
        rng = np.random.default_rng(D + N)
        nblk = N // bs + 3
        raw = torch.randint(-32768, 32768, (N, 2 * Hkv + 1, D), generator=_gen(N), device="cuda",
                            dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # every bit pattern, NaN too
        k, v = raw[:, :Hkv], raw[:, Hkv:2 * Hkv]
        slots = rng.permutation(nblk * bs)[:N]
        slots[rng.random(N) < 0.1] = -1
        slots[rng.random(N) < 0.05] = -(2 ** 40)
        pools = [_normal((nblk, Hkv, bs, D), 50 + i) for i in range(2)]
        ref = [bits(p) for p in pools]
        for r, src in zip(ref, (bits(k), bits(v))):
            for i, s in enumerate(slots):
                if s >= 0:
                    r[s // bs, :, s % bs] = src[i]
        g.kv_append_slots(*pools, k, v, torch.as_tensor(slots, device="cuda"))
        g.check_device_error()
        assert np.array_equal(bits(pools[0]), ref[0]) and np.array_equal(bits(pools[1]), ref[1])
        # past the pool: flagged, nothing else changes
        slots[0] = nblk * bs
        slots[N // 2] = 2 ** 62
        ref = [bits(p) for p in pools]
        g.kv_append_slots(*pools, k, v, torch.as_tensor(slots, device="cuda"))
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        assert np.array_equal(bits(pools[0]), ref[0]) and np.array_equal(bits(pools[1]), ref[1])


def test_append_slots_past_32_bits():
    # rows of a pool of more than 2^32 values, named by slots in its last block
    Hkv, bs, D = 8, 128, 128
    nblk = 2 ** 32 // (Hkv * bs * D) + 2
    pool = torch.zeros((nblk, Hkv, bs, D), dtype=torch.bfloat16, device="cuda")
    k, v = _normal((4, Hkv, D), 1), _normal((4, Hkv, D), 2)
    slots = torch.tensor([nblk * bs - 1, 3, (nblk - 1) * bs, nblk * bs - 2], device="cuda")
    vpool = torch.zeros_like(pool)
    g.kv_append_slots(pool, vpool, k, v, slots)
    g.check_device_error()
    assert torch.equal(pool[-1, :, -1], k[0]) and torch.equal(vpool[-1, :, 0], v[2])
    assert torch.equal(pool[-1, :, -2], k[3]) and torch.equal(pool[0, :, 3], k[1])
    del pool, vpool
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ 8-bit pool

def e4m3(x):
    """Nearest E4M3 value, ties to even, of |x| <= 448 (64-bit arithmetic)."""
    a = np.abs(x)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    e = np.where(np.exp2(e) > a, e - 1, np.where(np.exp2(e + 1) <= a, e + 1, e))
    step = np.exp2(np.maximum(e, -6) - 3)
    return np.copysign(np.round(a / step) * step, x)


CODE = np.array([torch.tensor([i], dtype=torch.uint8).view(torch.float8_e4m3fn).double().item() for i in range(256)])


def append8_ref(codes, scale, x, table, cached, cu, bs):
    """codes as values [nblk, Hkv, bs, D], scale [nblk, Hkv], x [N, Hkv, D], all float64."""
    val, sc = codes.copy(), scale.copy()
    for b in range(len(cached)):
        at, end, pos = cu[b], cu[b + 1], cached[b]
        while at < end:
            blk, r = table[b, pos // bs], pos % bs
            n = min(bs - r, end - at)
            rows = x[at:at + n].transpose(1, 0, 2)
            for h in range(x.shape[1]):
                a = np.abs(rows[h]).max()
                need = 2.0 ** -100
                if a > 0:
                    e = int(np.floor(np.log2(a))) - 10
                    while 448.0 * 2.0 ** e < a:
                        e += 1
                    need = 2.0 ** max(e, -100)
                now = max(need, sc[blk, h]) if r else need
                if r and now > sc[blk, h]:
                    val[blk, h, :r] = e4m3(val[blk, h, :r] * (sc[blk, h] / now))
                val[blk, h, r:r + n] = e4m3(rows[h] / now)
                sc[blk, h] = now
            at += n
            pos += n
    return val, sc


def make_table(lens, bs, seed, spare=2):
    nb = [-(-int(n) // bs) for n in lens]
    phys = np.random.default_rng(seed).permutation(sum(nb) + spare)
    table = np.full((len(lens), max(max(nb), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = phys[at:at + n]
        at += n
    return table, sum(nb) + spare


def values(codes):
    return CODE[codes.cpu().numpy()]


def new_pool8(nblk, Hkv, bs, D, seed):
    # every byte but E4M3's NaN, and any scales: a block that starts empty forgets them
    codes = torch.randint(0, 256, (nblk, Hkv, bs, D), generator=_gen(seed), device="cuda", dtype=torch.uint8)
    codes = torch.where((codes & 127) == 127, codes - 1, codes)
    scale = torch.full((nblk, Hkv), 2.0 ** 60, device="cuda")
    return codes.contiguous(), scale


def same_values(a, b):
    return np.array_equal(a, b)  # (-0 equals 0)


@pytest.mark.parametrize("D,Hkv,bs", [(64, 2, 16), (128, 1, 16), (128, 8, 64), (256, 2, 32), (64, 1, 1024),
                                      (128, 2, 128)])
def test_append8_step_after_step(D, Hkv, bs):
    rng = np.random.default_rng(D + bs)
    B = 6
    steps = [np.array([0, 1, 5, 40, bs, 2 * bs + 3]), np.ones(B, int), np.array([3, 0, 0, 17, 1, bs - 3]),
             np.ones(B, int), np.array([200, 1, 2, 3, 4, 5])]
    table, nblk = make_table(sum(steps), bs, D)
    pools = [new_pool8(nblk, Hkv, bs, D, 60 + i) for i in range(2)]
    refs = [(values(c), s.cpu().numpy().astype(np.float64)) for c, s in pools]
    cached = np.zeros(B, int)
    for i, new in enumerate(steps):
        cu = np.concatenate([[0], np.cumsum(new)])
        N = int(cu[-1]) + 2
        size = torch.exp2(torch.randint(-12, 13, (N, 1, 1), generator=_gen(i), device="cuda").float())
        kv = (_normal((N, 2 * Hkv, D), 70 + i).float() * size).to(torch.bfloat16)
        kv[rng.integers(0, N)] = 0
        k, v = kv[:, :Hkv], kv[:, Hkv:]
        g.kv_append_paged_fp8(pools[0][0], pools[1][0], pools[0][1], pools[1][1], k, v, _i32(table), _i32(cached),
                              _i32(cu))
        g.check_device_error()
        refs = [append8_ref(c, s, x.double().cpu().numpy(), table, cached, cu, bs) for (c, s), x in
                zip(refs, (k, v))]
        for (c, s), (rc, rs) in zip(pools, refs):
            assert np.array_equal(s.cpu().numpy().astype(np.float64), rs)
            assert same_values(values(c), rc)
        cached = cached + new


def test_append8_extremes():
    # the largest and smallest bf16 values, zeros, subnormals; scales from 2^-100 to 2^120
    D, Hkv, bs = 64, 1, 16
    big = float(torch.finfo(torch.bfloat16).max)
    sizes = [0.0, 2.0 ** -130, 2.0 ** -100, 448 * 2.0 ** -100, 450 * 2.0 ** -100, 1.75, 1.7578125, 448.0, 450.0, 1e30, big]
    table, nblk = make_table([len(sizes)], bs, 1)
    (kc, ks), (vc, vs) = new_pool8(nblk, Hkv, bs, D, 1), new_pool8(nblk, Hkv, bs, D, 2)
    ref = (values(kc), ks.cpu().numpy().astype(np.float64))
    for i, a in enumerate(sizes):
        x = torch.linspace(-1, 1, D, device="cuda").view(1, 1, D) * a
        x[0, 0, 0] = a
        x = x.to(torch.bfloat16)
        g.kv_append_paged_fp8(kc, vc, ks, vs, x, x, _i32(table), _i32([i]), _i32([0, 1]))
        g.check_device_error()
        ref = append8_ref(*ref, x.double().cpu().numpy(), table, [i], [0, 1], bs)
        assert np.array_equal(ks.cpu().numpy().astype(np.float64), ref[1])
        assert same_values(values(kc), ref[0])


def test_append8_bad_entries_between_good_ones():
    # blocks outside the pool between blocks inside, many heads in one block's turn
    D, Hkv, bs, nblk, B = 64, 8, 16, 300, 60
    rng = np.random.default_rng(8)
    table = rng.permutation(nblk)[:B * 5].reshape(B, 5).astype(np.int32)
    bad = rng.random((B, 5)) < 0.3
    t = np.where(bad, 1000, table)
    new = rng.integers(0, 5 * bs + 1, B)
    cu = np.concatenate([[0], np.cumsum(new)])
    kv = _normal((int(cu[-1]), 2 * Hkv, D), 3)
    pools = [new_pool8(nblk, Hkv, bs, D, 85 + i) for i in range(2)]
    refs = [(values(c), s.cpu().numpy().astype(np.float64)) for c, s in pools]
    g.kv_append_paged_fp8(pools[0][0], pools[1][0], pools[0][1], pools[1][1], kv[:, :Hkv], kv[:, Hkv:], _i32(t),
                          _i32([0] * B), _i32(cu))
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    for (c, s), (rc, rs), x in zip(pools, refs, (kv[:, :Hkv], kv[:, Hkv:])):
        wc, ws = append8_ref(rc, rs, x.double().cpu().numpy(), table, [0] * B, cu, bs)
        skipped = table[bad]
        wc[skipped], ws[skipped] = rc[skipped], rs[skipped]
        assert np.array_equal(s.cpu().numpy().astype(np.float64), ws)
        assert same_values(values(c), wc)


def test_append8_flags_and_skips_bad_requests():
    D, Hkv, bs, nblk = 128, 2, 16, 9
    table = np.array([[0, 1], [2, 99], [3, 4], [5, 6], [-1, 7]], np.int32)
    cached = np.array([3, 10, -1, 20, 0])
    cu = np.array([0, 5, 20, 25, 45, 50])  # request 1 runs into block 99, 3 past its row, 4 has no block
    kv = _normal((50, 2 * Hkv, D), 3)
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    pools = [new_pool8(nblk, Hkv, bs, D, 80 + i) for i in range(2)]
    refs = [(values(c), s.cpu().numpy().astype(np.float64)) for c, s in pools]
    g.kv_append_paged_fp8(pools[0][0], pools[1][0], pools[0][1], pools[1][1], k, v, _i32(table), _i32(cached), _i32(cu))
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    for (c, s), (rc, rs), x in zip(pools, refs, (k, v)):
        x = x.double().cpu().numpy()
        rc, rs = append8_ref(rc, rs, x, table, [3, 10], [0, 5, 11], bs)  # request 1's rows of block 2 alone
        assert np.array_equal(s.cpu().numpy().astype(np.float64), rs)
        assert same_values(values(c), rc)
    for bad in ([0, 60, 20, 25, 45, 50], [-3, 5, 20, 25, 45, 50], [0, 5, 2, 25, 45, 50]):
        g.kv_append_paged_fp8(pools[0][0], pools[1][0], pools[0][1], pools[1][1], k, v, _i32(np.abs(table) % nblk),
                              _i32([0] * 5), _i32(bad))
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)


def attn8_ref(q, kc, vc, ks, vs, table, lens, scale, bs):
    """(out, bound) in 64 bits.

    The bound: a weight times its scale is rounded to binary16 (2^-11) and
    enters as E4M3 parts whose unit keeps the largest scale's weight at 32 or
    more per unit of p, so that parts under half of E4M3's smallest step,
    2^-10, are lost: 2^-15 of the largest scale times |code|, per position, over
    a sum of weights of at least 1.  q enters as E4M3 parts, exact but for
    2^-17 of its largest |q| per entry, and scores of D products in fp32 add
    D 2^-24 sum|q k|: both move weights and their sum.  Last the bf16 output."""
    B, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    q, ks, vs = q.double().cpu().numpy(), ks.double().cpu().numpy(), vs.double().cpu().numpy()
    kcv, vcv = values(kc), values(vc)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = table[b, :-(-n // bs)]
        for h in range(Hkv):
            k = (kcv[ids, h] * ks[ids, h, None, None]).reshape(-1, D)[:n]
            v = (vcv[ids, h] * vs[ids, h, None, None]).reshape(-1, D)[:n]
            code = vcv[ids, h].reshape(-1, D)[:n]
            qs = q[b, h * G:(h + 1) * G]
            s = qs @ k.T * scale
            w = np.exp(s - s.max(1, keepdims=True))
            total = w.sum(1, keepdims=True)
            w = w / total
            o = w @ v
            ds = abs(scale) * (2.0 ** -17 * np.abs(qs).max(1, keepdims=True) * np.abs(k).sum(1).max()
                               + D * 2.0 ** -24 * (np.abs(qs) @ np.abs(k).T).max(1, keepdims=True))
            mag = w @ np.abs(v)
            lost = 2.0 ** -15 * vs[ids, h].max() * np.abs(code).sum(0) / total
            err = (2.0 ** -11 + 2 * ds + 2.0 ** -20) * mag + lost
            out[b, h * G:(h + 1) * G] = o
            bound[b, h * G:(h + 1) * G] = err + 2.0 ** -8 * (np.abs(o) + err)
    return out, bound


def run_attn8(lens, Hq, Hkv, D, bs, seed, scale=None):
    table, nblk = make_table(lens, bs, seed)
    kc, _ = new_pool8(nblk, Hkv, bs, D, seed)
    vc, _ = new_pool8(nblk, Hkv, bs, D, seed + 1)
    # values of about N(0, 1): scales a few powers of two around 2^-7, some not powers of two
    ks = torch.exp2(torch.randint(-9, -6, (nblk, Hkv), generator=_gen(seed), device="cuda").float()) * 1.25
    vs = torch.exp2(torch.randint(-9, -5, (nblk, Hkv), generator=_gen(seed + 2), device="cuda").float())
    used = np.zeros((nblk, bs), bool)
    for b, n in enumerate(lens):
        for i in range(-(-n // bs)):
            used[table[b, i], :min(bs, n - i * bs)] = True
    dead = torch.as_tensor(~used, device="cuda")[:, None, :].expand(nblk, Hkv, bs)
    kc[dead] = 0x7F  # NaN in every row that no position holds
    vc[dead] = 0xFF
    empty = torch.as_tensor(~used.any(1), device="cuda")
    ks[empty] = NAN
    vs[empty] = NAN
    q = _normal((len(lens), Hq, D), seed + 3)
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((len(lens), Hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    g.gqa_decode_attn_paged_fp8(q, kc, vc, ks, vs, _i32(table), _i32(lens), scale, out=out)
    g.check_device_error()
    ref, bound = attn8_ref(q, kc, vc, ks, vs, table, lens, scale, bs)
    o = out.double().cpu().numpy()
    assert np.isfinite(o).all()
    assert (np.abs(o - ref) <= bound).all(), float((np.abs(o - ref) - bound).max())


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 64, 8), (128, 8, 8), (128, 3, 1), (128, 48, 1), (128, 100, 1),
                                      (256, 16, 1), (256, 48, 1), (256, 6, 2)])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 1024])
def test_attn8_lengths_at_block_and_tile_edges(D, Hq, Hkv, bs):
    lens = sorted({0, 1, 2, bs - 1, bs, bs + 1, 127, 128, 129, 255, 256, 257, 3 * bs + 5, 1099} & set(range(1100)))
    run_attn8(lens, Hq, Hkv, D, bs, seed=bs + D + Hq)


@pytest.mark.parametrize("ctas", [1, 7, 300])
def test_attn8_small_and_large_grids(ctas):
    g.set_tuning(0, ctas)
    try:
        run_attn8([0, 900, 33, 1, 2048], 32, 4, 128, 16, seed=ctas)
        run_attn8([700, 0, 65], 16, 1, 256, 64, seed=ctas)
    finally:
        g.set_tuning(0, 0)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (128, 48, 1), (256, 16, 1)])
@pytest.mark.parametrize("ctas", [0, 3, 40])
def test_attn8_tile_counts_about_the_grid(D, Hq, Hkv, ctas):
    # one segment per head and many: fewer tiles than CTAs, as many, a few more,
    # and more pieces than a merge takes in a batch
    g.set_tuning(0, ctas)
    try:
        for n in (1, 2, 31, 33, 39, 40, 41, 79, 81, 161):
            run_attn8([128 * n - 5], Hq, Hkv, D, 64, seed=n)
        for n in (13, 14, 20, 40, 41, 152 // Hkv, 153 // Hkv + 1):
            run_attn8([0, 129] + [100] * n + [300], Hq, Hkv, D, 32, seed=n)
    finally:
        g.set_tuning(0, 0)


def test_attn8_graphs_of_one_stream_replay_side_by_side():
    # two graphs captured on one stream (the first calls there), with segments that
    # several CTAs share, replayed on two streams: each has a workspace of its own
    Hq, Hkv, D, bs = 16, 1, 128, 16
    g.release()
    stream, runs = torch.cuda.Stream(), []
    for seed, lens in ((1, [5000, 3000]), (2, [7000, 10])):
        table, nblk = make_table(lens, bs, seed)
        kc, ks = new_pool8(nblk, Hkv, bs, D, seed)
        vc, vs = new_pool8(nblk, Hkv, bs, D, seed + 10)
        ks.fill_(2.0 ** -8)
        vs.fill_(2.0 ** -8)
        q = _normal((2, Hq, D), seed)
        args = (q, kc, vc, ks, vs, _i32(table), _i32(lens), 0.1)
        out = torch.zeros((2, Hq, D), dtype=torch.bfloat16, device="cuda")
        want = g.gqa_decode_attn_paged_fp8(*args).clone()
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr, stream=stream):
            for _ in range(20):
                g.gqa_decode_attn_paged_fp8(*args, out=out)
        runs.append((gr, out, want, args))
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(30):
        for st, (gr, _, _, _) in zip(streams, runs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    g.check_device_error()
    for _, out, want, _ in runs:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_attn8_flags_bad_lengths_and_entries():
    Hq, Hkv, D, bs = 16, 2, 128, 16
    table, nblk = make_table([40, 40, 40], bs, 1)
    kc, ks = new_pool8(nblk, Hkv, bs, D, 1)
    vc, vs = new_pool8(nblk, Hkv, bs, D, 2)
    ks.fill_(2.0 ** -7)
    vs.fill_(2.0 ** -7)
    q = _normal((3, Hq, D), 3)
    ref, bound = attn8_ref(q, kc, vc, ks, vs, table, [40, 0, 40], 0.1, bs)
    for lens in ([40, -1, 40], [40, 3 * bs + 1, 40]):
        out = g.gqa_decode_attn_paged_fp8(q, kc, vc, ks, vs, _i32(table), _i32(lens), 0.1)
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    for entry in (-1, nblk, 2 ** 31 - 1):
        t = table.copy()
        t[1, 1] = entry
        out = g.gqa_decode_attn_paged_fp8(q, kc, vc, ks, vs, _i32(t), _i32([40, 40, 40]), 0.1)
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        o = out.double().cpu().numpy()
        assert (np.abs(o - ref) <= bound)[[0, 2]].all()


# --------------------------------------------------------------- the whole path

@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (256, 16, 1)])
@pytest.mark.parametrize("order", [1, -1, 0])
def test_attn8_scales_far_apart(D, Hq, Hkv, order):
    # value scales that rise, fall or jump over 200 binary orders from block to
    # block (the unit of the weights has to follow), zeros and a single head
    # without any; key scales of zero
    bs, lens = 16, [700, 16, 130, 1]
    table, nblk = make_table(lens, bs, 5)
    kc, _ = new_pool8(nblk, Hkv, bs, D, 6)
    vc, _ = new_pool8(nblk, Hkv, bs, D, 7)
    ks = torch.full((nblk, Hkv), 2.0 ** -8, device="cuda")
    vs = torch.zeros((nblk, Hkv), device="cuda")
    rng = np.random.default_rng(8)
    for b, n in enumerate(lens):
        ids = torch.as_tensor(table[b, :-(-n // bs)].astype(np.int64), device="cuda")
        e = np.linspace(-100, 100, len(ids))
        e = rng.permutation(e) if order == 0 else e[::order].copy()
        vs[ids] = torch.exp2(torch.as_tensor(np.round(e), device="cuda").float())[:, None]
        vs[ids[len(ids) // 2:][:1], 0] = 0.0
        ks[ids[:2], Hkv - 1] = 0.0
    q = _normal((len(lens), Hq, D), 9)
    out = torch.full((len(lens), Hq, D), NAN, dtype=torch.bfloat16, device="cuda")
    g.gqa_decode_attn_paged_fp8(q, kc, vc, ks, vs, _i32(table), _i32(lens), 1 / math.sqrt(D), out=out)
    g.check_device_error()
    ref, bound = attn8_ref(q, kc, vc, ks, vs, table, lens, 1 / math.sqrt(D), bs)
    o = out.double().cpu().numpy()
    assert np.isfinite(o).all()
    assert (np.abs(o - ref) <= bound).all()


def test_attn8_requests_that_share_blocks():
    # one prefix's blocks in many table rows, read to different lengths
    bs, Hkv, D = 16, 2, 128
    table, nblk = make_table([400], bs, 3)
    kc, _ = new_pool8(nblk, Hkv, bs, D, 1)
    vc, _ = new_pool8(nblk, Hkv, bs, D, 2)
    ks, vs = (torch.full((nblk, Hkv), 2.0 ** -7, device="cuda") for _ in range(2))
    lens = [400, 399, 128, 129, 1, 0, 400]
    table = np.repeat(table, len(lens), 0)
    q = _normal((len(lens), 16, D), 4)
    out = g.gqa_decode_attn_paged_fp8(q, kc, vc, ks, vs, _i32(table), _i32(lens), 0.1)
    g.check_device_error()
    ref, bound = attn8_ref(q, kc, vc, ks, vs, table, lens, 0.1, bs)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_pool8_past_32_bits():
    bs, D, nblk = 1024, 256, 16400  # 4.3 GB of K codes, as many of V
    codes = [torch.zeros((nblk, 1, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((nblk, 1), device="cuda") for _ in range(2)]
    table = np.array([[nblk - 1, 16384, 0], [16383, 1, 2]], np.int32)  # block 16384 starts at byte 2^32
    lens, cu = [2100, 700], [0, 2100, 2800]
    q = _normal((2, 16, D), 1)
    k, v = (_normal((2800, 1, D), i) for i in (2, 3))
    g.kv_append_paged_fp8(*codes, *scales, k, v, _i32(table), _i32([0, 0]), _i32(cu))
    out = g.gqa_decode_attn_paged_fp8(q, *codes, *scales, _i32(table), _i32(lens), 1 / 16)
    g.check_device_error()
    ids = table.ravel()
    at = torch.as_tensor(ids.astype(np.int64), device="cuda")
    kc, vc = (c[at] for c in codes)
    ks, vs = (s[at] for s in scales)
    near = np.arange(6, dtype=np.int32).reshape(2, 3)
    for c, s, x in ((kc, ks, k), (vc, vs, v)):
        empty = np.zeros((6, 1, bs, D))
        rc, rs = append8_ref(empty, np.zeros((6, 1)), x.double().cpu().numpy(), near, [0, 0], cu, bs)
        used = [0, 1, 2, 3]
        assert np.array_equal(s.cpu().numpy()[used], rs[used])
        assert same_values(values(c)[used], rc[used])
    assert not any(bool(c[5].any()) for c in codes)
    ref, bound = attn8_ref(q, kc, vc, ks, vs, near, lens, 1 / 16, bs)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    del codes
    torch.cuda.empty_cache()


def test_attn8_schedule_past_32_bits():
    # so many segments that their cost passes 2^31; all read one block's first row
    B, H, D, bs = 65535, 384, 128, 16
    codes = torch.randint(0, 120, (1, H, bs, D), generator=_gen(1), device="cuda", dtype=torch.uint8)
    scale = torch.full((1, H), 0.25, device="cuda")
    q = torch.ones((B, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full((B, H, D), NAN, dtype=torch.bfloat16, device="cuda")
    g.gqa_decode_attn_paged_fp8(q, codes, codes, scale, scale, torch.zeros((B, 1), dtype=torch.int32, device="cuda"),
                                torch.ones(B, dtype=torch.int32, device="cuda"), 0.1, out=out)
    g.check_device_error()
    row = (codes[0, :, 0].view(torch.float8_e4m3fn).float() * 0.25).to(torch.bfloat16)
    assert bool((out == row).all())
    del q, out
    torch.cuda.empty_cache()


def test_the_largest_batch():
    # 65535 requests of one token each: attention gives its value row back, exactly
    # (a weight of one; a power of two times a code)
    B, D, bs = 65535, 128, 16
    zeros = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(B, dtype=torch.int32, device="cuda")
    cu, slots, left = g.kv_block_tables(zeros, zeros + 1, table, free, _i32([B]), bs, B + 1)
    g.check_device_error()
    want = torch.arange(B - 1, -1, -1, device="cuda")
    assert int(left) == 0 and torch.equal(table[:, 0].long(), want)
    assert torch.equal(cu.long(), torch.arange(B + 1, device="cuda"))
    assert torch.equal(slots[:B], want * bs) and int(slots[B]) == -1

    q, k, v = (_normal((B, 1, D), i) for i in range(3))
    out = g.gqa_prefill_attn(q, k, v, cu, 0.1)
    g.check_device_error()
    assert torch.equal(out, v)

    codes = [torch.zeros((B, 1, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((B, 1), device="cuda") for _ in range(2)]
    g.kv_append_paged_fp8(*codes, *scales, k, v, table, zeros, cu)
    g.check_device_error()
    for c, s, x in zip(codes, scales, (k, v)):
        x = x[:, 0].double()
        need = torch.exp2(torch.ceil(torch.log2(x.abs().amax(1) / 448)))
        assert torch.equal(s[want, 0].double(), need)
        rows = (x / need[:, None]).to(torch.float32).to(torch.float8_e4m3fn)
        assert torch.equal(c[want, 0, 0].view(torch.float8_e4m3fn).float(), rows.float())
    out = g.gqa_decode_attn_paged_fp8(q, *codes, *scales, table, zeros + 1, 0.1)
    g.check_device_error()
    row = codes[1][want, 0, 0].view(torch.float8_e4m3fn).float() * scales[1][want]
    assert torch.equal(out[:, 0].float(), row)


def test_prompts_then_steps_through_bf16_and_8_bit_pools():
    """Admission, prompt attention and single-token steps: after each step the
    pools hold the tokens' rows and decode attention sees all of them."""
    B, Hq, Hkv, D, bs, nblk, maxb = 5, 16, 2, 128, 16, 80, 12
    scale = 1 / math.sqrt(D)
    table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(nblk, generator=_gen(0), device="cuda").to(torch.int32)
    count = _i32([nblk])
    k_pool, v_pool = (torch.full((nblk, Hkv, bs, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc, vc = (torch.full((nblk, Hkv, bs, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((nblk, Hkv), NAN, device="cuda") for _ in range(2))
    have = [0] * B
    all_k, all_v = [[] for _ in range(B)], [[] for _ in range(B)]
    for step, new in enumerate(([37, 0, 16, 1, 100], [1, 70, 1, 1, 1], [1, 1, 1, 1, 1], [0, 1, 0, 1, 20])):
        total = sum(new)
        qkv = _normal((total + 2, Hq + 2 * Hkv, D), 90 + step)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        cu, slots, _ = g.kv_block_tables(_i32(have), _i32(new), table, free, count, bs, total + 2)
        g.kv_append_slots(k_pool, v_pool, k, v, slots)
        g.kv_append_paged_fp8(kc, vc, ks, vs, k, v, table, _i32(have), cu)
        g.check_device_error()
        cu_h = cu.cpu().tolist()
        out = g.gqa_prefill_attn(q, k, v, cu, scale)
        check_prefill(out[:total], *(x[:total] for x in prefill_ref(q, k, v, cu_h, scale)))
        for b in range(B):
            all_k[b].append(k[cu_h[b]:cu_h[b + 1]])
            all_v[b].append(v[cu_h[b]:cu_h[b + 1]])
            have[b] += new[b]
        # the last token of every request over its whole cache
        qd = _normal((B, Hq, D), 95 + step)
        lens = _i32(have)
        o16 = g.gqa_decode_attn_paged(qd, k_pool, v_pool, table, lens, scale)
        o8 = g.gqa_decode_attn_paged_fp8(qd, kc, vc, ks, vs, table, lens, scale)
        g.check_device_error()
        th = table.cpu().numpy()
        ref8, bound8 = attn8_ref(qd, kc, vc, ks, vs, th, have, scale, bs)
        assert (np.abs(o8.double().cpu().numpy() - ref8) <= bound8).all()
        for b in range(B):
            if have[b] == 0:
                assert not o16[b].any() and not o8[b].any()
                continue
            kb, vb = torch.cat(all_k[b]).double(), torch.cat(all_v[b]).double()
            for h in range(Hq):
                w = torch.softmax(qd[b, h].double() @ kb[:, h // 8].T * scale, 0)
                ref = w @ vb[:, h // 8]
                assert float((o16[b, h].double() - ref).abs().max()) <= 2e-3
                # E4M3 rows are off by 2^-4 of themselves at most (or, small ones, by
                # 2^-10 of a scale that is at most 2^-7 here): K moves a score by
                # 2^-4 scale sum|q k|, so compare loosely: the pool holds these rows
                assert float((o8[b, h].double() - ref).abs().max()) <= 0.6
    used = sorted(int(x) for row in table.cpu() for x in row if x >= 0)
    assert len(set(used)) == len(used) == nblk - int(count)


def test_calls_on_another_stream_than_the_current_one():
    # outputs that a call makes belong to its stream: nothing of the current
    # stream, busy here, may come behind them
    side = torch.cuda.Stream()
    qkv = _normal((200, 10, 128), 1)
    q, k, v = qkv[:, :8], qkv[:, 8:9], qkv[:, 9:]
    last = qkv[[149, 199], :8].contiguous()
    cu, cached, new = _i32([0, 150, 200]), _i32([0, 0]), _i32([150, 50])
    for busy in (False, True):  # (a first call may wait for the device by itself)
        table, free, count = torch.full((2, 16), -1, dtype=torch.int32, device="cuda"), _i32(range(20)), _i32([20])
        pool = [torch.zeros((20, 1, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((20, 1), device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(200_000_000)  # some 0.1 s
        out = g.gqa_prefill_attn(q, k, v, cu, 0.1, stream=side)
        rows, slots, left = g.kv_block_tables(cached, new, table, free, count, 16, 200, stream=side)
        g.kv_append_paged_fp8(*pool, *scales, k, v, table, cached, rows, stream=side)
        step = g.gqa_decode_attn_paged_fp8(last, *pool, *scales, table, new, 0.1, stream=side)
        torch.cuda.synchronize()
        g.check_device_error()
        check_prefill(out, *prefill_ref(q, k, v, [0, 150, 200], 0.1))
        assert rows.tolist() == [0, 150, 200] and int(left) == 20 - 10 - 4 and int((slots < 0).sum()) == 0
        ref, bound = attn8_ref(last, *pool, *scales, table.cpu().numpy(), [150, 50], 0.1, 16)
        assert (np.abs(step.double().cpu().numpy() - ref) <= bound).all()


def test_a_stream_is_anything_with_its_handle():
    class Handle:
        cuda_stream = torch.cuda.Stream().cuda_stream

    qkv = _normal((40, 3, 64), 1)
    torch.cuda.synchronize()
    out = g.gqa_prefill_attn(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], _i32([0, 40]), 0.1, stream=Handle())
    torch.cuda.synchronize()
    g.check_device_error()
    check_prefill(out, *prefill_ref(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], [0, 40], 0.1))


def test_the_path_captured_and_replayed():
    """One decode step of every call in a graph, replayed: lengths and the free
    list advance on the device."""
    B, Hq, Hkv, D, bs, nblk = 4, 8, 2, 128, 16, 40
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(nblk, dtype=torch.int32, device="cuda")
    count, lens, one = _i32([nblk]), _i32([0] * B), _i32([1] * B)
    kc, vc = (torch.zeros((nblk, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nblk, Hkv), device="cuda") for _ in range(2))
    kp, vp = (torch.zeros((nblk, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = _normal((B, Hq, D), 1), _normal((B, Hkv, D), 2), _normal((B, Hkv, D), 3)
    cu, slots = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    out = torch.zeros((B, Hq, D), dtype=torch.bfloat16, device="cuda")
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        g.kv_block_tables(lens, one, table, free, count, bs, B, cu_seqlens=cu, slots=slots)
        g.kv_append_slots(kp, vp, k, v, slots)
        g.kv_append_paged_fp8(kc, vc, ks, vs, k, v, table, lens, cu)
        lens.add_(1)
        g.gqa_decode_attn_paged_fp8(q, kc, vc, ks, vs, table, lens, 0.1, out=out)
    rows = []
    for step in range(40):
        k.copy_(_normal((B, Hkv, D), 100 + step))
        v.copy_(_normal((B, Hkv, D), 200 + step))
        rows.append(v.clone())
        gr.replay()
        torch.cuda.synchronize()
        if step in (0, 15, 16, 39):
            g.check_device_error()
            th = table.cpu().numpy()
            ref, bound = attn8_ref(q, kc, vc, ks, vs, th, [step + 1] * B, 0.1, bs)
            assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
            assert int(count) == nblk - B * (step // bs + 1)
            for b in range(B):
                blk = int(th[b, step // bs])
                assert torch.equal(vp[blk, :, step % bs], rows[step][b])


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (128, 48, 1), (256, 16, 1)])
@pytest.mark.parametrize("captured", [False, True])
def test_attention_before_an_append_that_rewrites_its_blocks(D, Hq, Hkv, captured):
    # requests of one tile, so that no segment is split and the merge has nothing
    # to do; the append behind it overwrites every row that the attention reads,
    # and each attention call writes the output of the one before it
    bs, lens, turns = 16, [100, 128, 33, 64], 40
    table, nblk = make_table(lens, bs, D)
    cu = np.concatenate([[0], np.cumsum(lens)])
    slots = torch.as_tensor(np.concatenate([table[b, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
                                            for b, n in enumerate(lens)]), device="cuda")
    q = _normal((len(lens), Hq, D), 1)
    rows = [(_normal((cu[-1], Hkv, D), 10 + i), _normal((cu[-1], Hkv, D), 20 + i)) for i in range(3)]
    d_table, d_lens, d_cu, zero = _i32(table), _i32(lens), _i32(cu), _i32([0] * len(lens))

    def run(settle):
        codes = [torch.zeros((nblk, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((nblk, Hkv), device="cuda") for _ in range(2)]
        pools = [torch.zeros((nblk, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        outs8 = [torch.zeros((len(lens), Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(turns)]
        outs16 = [torch.zeros((len(lens), Hq, D), device="cuda") for _ in range(turns)]

        def steps():
            for i in range(turns):
                k, v = rows[i % 3]
                g.kv_append_paged_fp8(*codes, *scales, k, v, d_table, zero, d_cu)
                settle()
                g.gqa_decode_attn_paged_fp8(q, *codes, *scales, d_table, d_lens, 0.1, out=outs8[i])
                settle()
            for i in range(turns):
                g.kv_append_slots(*pools, *rows[i % 3], slots)
                settle()
                g.gqa_decode_attn_paged(q, *pools, d_table, d_lens, 0.1, out=outs16[i])
                settle()

        if captured and settle is not torch.cuda.synchronize:
            g.gqa_decode_attn_paged(q, *pools, d_table, d_lens, 0.1)  # (its workspace is there before the capture)
            gr, stream = torch.cuda.CUDAGraph(), torch.cuda.current_stream()
            side = torch.cuda.Stream()
            side.wait_stream(stream)
            with torch.cuda.stream(side):
                g.gqa_decode_attn_paged(q, *pools, d_table, d_lens, 0.1)
            torch.cuda.synchronize()
            with torch.cuda.graph(gr, stream=side):
                steps()
            gr.replay()
        else:
            torch.cuda.synchronize()
            steps()
        torch.cuda.synchronize()
        g.check_device_error()
        return outs8 + outs16

    for a, b in zip(run(torch.cuda.synchronize), run(lambda: None)):
        assert torch.equal(a, b)


def _split_call(lens, seed, Hq=16, Hkv=1, D=128, bs=16):
    """Arguments of a paged 8-bit call whose segments several CTAs share."""
    table, nblk = make_table(lens, bs, seed)
    kc, ks = new_pool8(nblk, Hkv, bs, D, seed)
    vc, vs = new_pool8(nblk, Hkv, bs, D, seed + 10)
    ks.fill_(2.0 ** -8)
    vs.fill_(2.0 ** -8)
    return _normal((len(lens), Hq, D), seed), kc, vc, ks, vs, _i32(table), _i32(lens), 0.1


def test_attn8_workspaces_of_captures_go_with_their_graphs():
    # graphs captured anew for ever, a few alive at a time: device memory does not
    # grow, and the ones alive keep their workspaces to themselves
    g.release()
    calls = [_split_call(lens, seed) for seed, lens in ((1, [5000, 3000]), (2, [700] * 60), (3, [6000]))]
    wants = [g.gqa_decode_attn_paged_fp8(*c).clone() for c in calls]
    outs = [torch.zeros_like(w) for w in wants]
    stream, alive = torch.cuda.Stream(), []

    def turn(i):
        which = [i % 3, (i + i // 3) % 3]  # (a second call may need a larger one)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=stream):
            for j in which:
                g.gqa_decode_attn_paged_fp8(*calls[j], out=outs[j])
        alive.append((gr, which))
        if len(alive) > 4:
            alive.pop(0)
        for gr, which in alive:
            for o in outs:
                o.fill_(7.0)
            gr.replay()
            torch.cuda.synchronize()
            for j in which:
                assert torch.equal(outs[j].view(torch.int16), wants[j].view(torch.int16))

    for i in range(24):
        turn(i)
    free = torch.cuda.mem_get_info()[0]
    for i in range(24, 120):
        turn(i)
    lost = free - torch.cuda.mem_get_info()[0]
    g.check_device_error()
    assert lost < 16 << 20, lost  # (96 captures with a workspace of 1 MB or more each)


def test_attn8_release_between_captures():
    call = _split_call([4000, 100], 4)
    want = g.gqa_decode_attn_paged_fp8(*call).clone()
    out = torch.zeros_like(want)
    stream, old = torch.cuda.Stream(), []
    for i in range(6):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=stream):
            g.gqa_decode_attn_paged_fp8(*call, out=out)
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        g.check_device_error()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        g.release()       # its workspace is gone: not replayed again,
        old.append(gr)    # only destroyed, at once or after the next capture
        if i % 2:
            old.clear()


def test_windows_beyond_32_bits():
    # past every position: the full attention; below 1: refused; never the low bits
    n, D = 300, 128
    q, k, v = _normal((n, 8, D), 1), _normal((n, 2, D), 2), _normal((n, 2, D), 3)
    kc, vc = (t.transpose(0, 1).contiguous()[None] for t in (k, v))
    table = _i32([[0, 1, 2]])
    kp, vp = (torch.zeros((3, 2, 128, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g.kv_append_slots(kp, vp, k, v, torch.arange(n, device="cuda"))
    lens, before = _i32([n]), _i32([n - 1])
    calls = [lambda w: g.gqa_prefill_attn(q, k, v, _i32([0, n]), 0.1, window=w),
             lambda w: g.gqa_decode_attn(q[:1], kc, vc, lens, 0.1, window=w),
             lambda w: g.gqa_decode_step(q[:1], k[-1:], v[-1:], kc, vc, before, 0.1, window=w),
             lambda w: g.gqa_decode_attn_multi(q[None, :2], kc, vc, lens, 0.1, window=w),
             lambda w: g.gqa_decode_attn_paged(q[:1], kp, vp, table, lens, 0.1, window=w),
             lambda w: g.gqa_decode_step_paged(q[:1], k[-1:], v[-1:], kp, vp, table, before, 0.1, window=w)]
    for call in calls:
        full = call(n + 1)
        assert not torch.equal(call(5), full)
        for w in (2 ** 31, 2 ** 32 + 5, 2 ** 40):
            assert torch.equal(call(w), full)
        for w in (0, -5, -2 ** 31, -2 ** 32 + 5, -2 ** 40):
            with pytest.raises(g.KvAttnError) as ei:
                call(w)
            assert ei.value.status == g.KVATTN_ERR_INVALID_ARG
    g.check_device_error()
