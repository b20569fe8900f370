"""GPU parity of the attention of packed tokens over a paged pool: tokens that
continue what their request has cached (gqa_extend_attn) and tokens over an
encoder's states (gqa_cross_attn), against the definition in 64 bits.

Tolerance, as for prompt attention: a weight is rounded to bf16 (2^-8 of it), the
result once more (2^-8 of it); a score of D products in fp32 is off by at most
D 2^-24 sum|q k| scale, which with N(0,1) inputs stays under 2^-11 together with
the weights' sum, and joining pieces adds a few 2^-24.  So
|out - ref| <= (2^-8 + 2^-10) sum_j w_j |v_j| + 2^-8 |out|.
"""
import math

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


class Case:
    """A pool, its table and packed queries; what no token attends is poisoned."""

    def __init__(self, new, kv, Hq, Hkv, D, bs, seed, causal=True, window=None, gap=0, pad=3, wide=True, spare=3):
        self.new, self.kv, self.Hq, self.Hkv, self.D, self.bs = new, kv, Hq, Hkv, D, bs
        self.causal, self.window = causal, window
        self.scale = 1 / math.sqrt(D)
        starts = [gap]
        for n in new:
            starts.append(starts[-1] + n)
        self.starts, N = starts, starts[-1] + pad
        q = _normal((N, Hq + (2 if wide else 0), D), seed)
        self.q = q[:, 1:Hq + 1] if wide else q
        self.q[:gap] = NAN
        self.q[starts[-1]:] = NAN
        nb = [-(-n // bs) for n in kv]
        nblk = max(1, sum(nb) + spare)
        ids = torch.randperm(nblk, generator=torch.Generator().manual_seed(seed))
        self.table = torch.full((len(kv), max(1, max(nb)) + 1), -1, dtype=torch.int64)
        k, v = _normal((nblk, Hkv, bs, D), seed + 1), _normal((nblk, Hkv, bs, D), seed + 2)
        self.k_pool, self.v_pool = torch.full_like(k, NAN), torch.full_like(v, NAN)
        at = 0
        for b, n in enumerate(kv):
            self.table[b, :nb[b]] = ids[at:at + nb[b]]
            at += nb[b]
            lo, hi = self.span(b)
            for e in range(nb[b]):
                i = int(self.table[b, e])
                a, z = max(lo - e * bs, 0), min(hi - e * bs, bs)
                if a < z:
                    for pool, x in ((self.k_pool, k), (self.v_pool, v)):
                        pool[i, :, a:z] = x[i, :, a:z]
                else:  # nobody attends it
                    self.table[b, e] = -1 - e
        self.args = (self.q, self.k_pool, self.v_pool, _i32(self.table), _i32(kv), _i32(starts), self.scale)

    def span(self, b):
        """Positions that some token of sequence b attends."""
        if not self.new[b]:
            return 0, 0
        first = self.ends(b)[0]
        return (max(0, max(first, 1) - self.window) if self.window else 0), self.kv[b]

    def ends(self, b):
        n, m = self.new[b], self.kv[b]
        return [m - n + i + 1 for i in range(n)] if self.causal else [m] * n

    def run(self, out=None, **more):
        if self.causal:
            return g.gqa_extend_attn(*self.args, out=out, window=self.window, **more)
        return g.gqa_cross_attn(*self.args, out=out, **more)

    def ref(self):
        """(result, sum of weights times |v|) in 64 bits; NaN in rows of no sequence."""
        N, G = self.q.shape[0], self.Hq // self.Hkv
        out = torch.full((N, self.Hq, self.D), NAN, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(out)
        for b, m in enumerate(self.kv):
            a, e = self.starts[b], self.starts[b + 1]
            if a == e:
                continue
            lo, hi = self.span(b)
            ids = self.table[b, :-(-m // self.bs)].clamp(min=0).cuda()
            out[a:e] = 0
            if not m:
                continue
            k, v = (p[ids].double().permute(1, 0, 2, 3).reshape(self.Hkv, -1, self.D)[:, lo:hi]
                    for p in (self.k_pool, self.v_pool))
            end = torch.tensor(self.ends(b), device="cuda")[:, None]
            j = torch.arange(lo, hi, device="cuda")[None, :]
            hidden = j >= end
            if self.window:
                hidden |= j < end - self.window
            some = (~hidden).any(1)
            q = self.q[a:e].double().permute(1, 0, 2)
            for h in range(self.Hq):
                s = q[h] @ k[h // G].T * self.scale
                s = s.masked_fill(hidden, -math.inf)[some]
                w = torch.softmax(s, 1)
                out[a:e, h][some] = w @ v[h // G]
                mag[a:e, h][some] = w @ v[h // G].abs()
        return out, mag

    def check(self, out=None, before=None, ref=None):
        if out is None:
            before = torch.full((self.q.shape[0], self.Hq, self.D), 7.25, dtype=torch.bfloat16, device="cuda")
            out = self.run(out=before.clone())
            g.check_device_error()
        ref, mag = ref or self.ref()
        mine = ~torch.isnan(ref[:, 0, 0])
        o = out.double()
        assert bool(torch.isfinite(o[mine]).all())
        over = (o - ref)[mine].abs() - ((2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * o.abs())[mine]
        assert not over.numel() or float(over.max()) <= 0, float(over.max())
        if before is not None:
            assert torch.equal(out[~mine].view(torch.int16), before[~mine].view(torch.int16))
        return out


HEADS = [(64, 4, 4), (64, 6, 2), (64, 3, 1), (128, 64, 8), (128, 8, 8), (128, 5, 1), (128, 32, 1), (256, 16, 1),
         (256, 48, 1), (256, 3, 1), (256, 4, 4), (128, 256, 1), (64, 7, 1)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_one_token(D, Hq, Hkv, causal):
    for kv in (1, 16, 17, 128, 300):
        Case([1], [kv], Hq, Hkv, D, 16, seed=kv, causal=causal, pad=0).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_a_step_of_single_tokens(D, Hq, Hkv, causal):
    kv = [1, 15, 16, 17, 0, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700, 1025, 2, 40]
    Case([1] * len(kv), kv, Hq, Hkv, D, 32, seed=D + Hq, causal=causal).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_ragged_counts_over_ragged_lengths(D, Hq, Hkv, causal):
    new = [0, 1, 2, 5, 16, 17, 1, 0, 33, 64, 100, 128, 129, 1, 200, 300, 3, 0]
    old = [9, 0, 126, 3, 0, 120, 999, 5, 128, 64, 29, 128, 1, 512, 57, 400, 254, 0]
    kv = [n + o for n, o in zip(new, old)] if causal else [o * 2 for o in old]
    Case(new, kv, Hq, Hkv, D, 64, seed=D + Hq, causal=causal, gap=5).check()


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 16), (128, 64, 8), (256, 16, 1)])
def test_block_sizes(D, Hq, Hkv, bs):
    Case([1, 70, 300, 1], [700, 71, 900, 16], Hq, Hkv, D, bs, seed=bs).check()
    Case([1, 70, 300, 1], [700, 71, 900, 16], Hq, Hkv, D, bs, seed=bs, causal=False).check()


@pytest.mark.parametrize("window", [1, 5, 16, 100, 127, 128, 129, 300, 5000])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 64, 8), (128, 3, 1), (256, 16, 1)])
def test_windows(D, Hq, Hkv, window):
    # (blocks that nobody attends are not in the table, and rows nobody attends are NaN)
    new = [1, 300, 70, 1, 513, 2]
    kv = [900, 300, 400, 130, 1200, 129]
    Case(new, kv, Hq, Hkv, D, 16, seed=window, window=window).check()


@pytest.mark.parametrize("ctas", [1, 2, 7, 40, 151])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 64, 8), (256, 16, 1)])
def test_any_number_of_ranges(D, Hq, Hkv, ctas):
    g.set_tuning(0, ctas)
    try:
        Case([1, 300, 2, 0, 1, 150], [2500, 1400, 2, 9, 1, 3001], Hq, Hkv, D, 64, seed=ctas).check()
        Case([1, 300, 2, 5, 1], [2500, 1400, 2, 0, 130], Hq, Hkv, D, 64, seed=ctas, causal=False).check()
        Case([200, 1], [3000, 2000], Hq, Hkv, D, 64, seed=ctas, window=700).check()
    finally:
        g.set_tuning(0, 0)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 8, 1), (256, 16, 1), (256, 1, 1)])
def test_one_long_request_over_all_ranges(D, Hq, Hkv):
    Case([1], [60_000], Hq, Hkv, D, 64, seed=D, pad=0).check()
    Case([3], [50_001], Hq, Hkv, D, 16, seed=D, causal=False).check()


def test_more_tokens_than_positions():
    # the tokens at negative positions attend nothing
    Case([5, 300, 3], [3, 100, 0], 8, 2, 128, 16, seed=1).check()
    Case([5, 300, 3], [3, 100, 0], 4, 1, 256, 16, seed=1, window=20).check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30, 1.0, 3.0])
def test_scales(scale):
    c = Case([40, 1], [300, 200], 8, 2, 128, 32, seed=3)
    c.scale = scale
    c.q.mul_(0.25)  # (scores of a few units at scale 3)
    c.args = c.args[:-1] + (scale,)
    c.check()


def test_scores_that_grow_along_the_keys_move_the_maximum():
    c = Case([130, 1], [1500, 1300], 8, 2, 128, 64, seed=4)
    for b in range(2):
        for e, i in enumerate(c.table[b, :-(-c.kv[b] // 64)].tolist()):
            c.k_pool[i] *= 0.2 + e / 4
    # (scores up to 6 * sum|q k| scale: fp32 carries them to 2^-24 * 128 * 60)
    c.check()


@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("causal,window", [(True, None), (True, 1), (True, 100), (True, 700), (False, None)])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (64, 8, 1), (128, 64, 8), (128, 3, 1), (256, 16, 1), (256, 2, 2)])
def test_few_tokens_on_average_and_some_of_many(D, Hq, Hkv, causal, window, bs):
    # (units of few rows and of many in one call, in every order)
    new = [1, 300, 1, 2, 0, 1, 70, 1, 1, 3, 129, 1, 4, 31, 1, 33, 8, 1] + [0] * 300
    old = [2000, 100, 127, 128, 5, 0, 600, 129, 383, 1, 0, 1300, 255, 7, 1, 0, 77, 640] + [0, 17] * 150
    kv = [n + o for n, o in zip(new, old)] if causal else old
    c = Case(new, kv, Hq, Hkv, D, bs, seed=bs + D, causal=causal, window=window)
    ref = c.ref()
    for ctas in (0, 1, 3, 40):
        g.set_tuning(0, ctas)
        try:
            before = torch.full((c.q.shape[0], Hq, D), 7.25, dtype=torch.bfloat16, device="cuda")
            out = c.run(out=before.clone())
            g.check_device_error()
            c.check(out, before, ref)
        finally:
            g.set_tuning(0, 0)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 16), (128, 64, 8), (128, 20, 1), (256, 16, 1), (256, 32, 1)])
def test_steps_back_to_back(D, Hq, Hkv):
    cases = [Case([1] * 40, [(37 * i + 11 * s) % 900 + 1 for i in range(40)], Hq, Hkv, D, 16, seed=s) for s in range(3)]
    outs = [c.run() for _ in range(10) for c in cases]
    g.check_device_error()
    for i, c in enumerate(cases):
        ref = c.ref()
        for o in outs[i::3]:
            c.check(o, ref=ref)
            assert torch.equal(o[:40], outs[i][:40])


def test_heads_that_fill_no_power_of_two():
    for Hq, Hkv, D in ((96, 1, 128), (130, 1, 64), (24, 2, 128), (200, 2, 256), (33, 1, 128), (18, 6, 64)):
        Case([1, 1, 2, 0], [300, 129, 77, 5], Hq, Hkv, D, 16, seed=Hq).check()
        Case([40, 1, 150], [300, 129, 200], Hq, Hkv, D, 64, seed=Hq, causal=False).check()


def test_many_sequences_most_of_them_empty():
    rng = np.random.RandomState(1)
    new = [0] * 3000
    kv = [0] * 3000
    for b in rng.choice(3000, 70, replace=False):
        new[b] = int(rng.randint(1, 40))
        kv[b] = new[b] + int(rng.randint(0, 600))
    for b in rng.choice(3000, 40, replace=False):
        kv[b] = max(kv[b], 33)  # lengths without tokens
    Case(new, kv, 8, 2, 128, 16, seed=2).check()
    Case(new, kv, 2, 1, 256, 16, seed=2, causal=False).check()


def test_the_same_bits_every_time_and_rows_that_two_tables_share():
    c = Case([1, 200, 60], [3000, 900, 60], 64, 8, 128, 64, seed=6)
    first = c.check()[:261]  # (the rows behind are not written)
    for _ in range(5):
        assert torch.equal(c.run()[:261], first)
    # rows shared by two sequences' tables (an encoder's states of two forks)
    c = Case([7, 7], [300, 300], 8, 2, 128, 16, seed=7, causal=False)
    c.table[1] = c.table[0]
    c.args = c.args[:3] + (_i32(c.table),) + c.args[4:]
    c.check()


def test_it_is_prompt_attention_where_nothing_is_cached_and_decode_where_one_is_new():
    Hq, Hkv, D, bs = 16, 4, 128, 16
    lens = [70, 1, 200]
    c = Case(lens, lens, Hq, Hkv, D, bs, seed=8, pad=0, wide=False)
    out = c.check()
    k, v = (torch.cat([p[c.table[b, :-(-n // bs)].cuda()].permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:n]
                       for b, n in enumerate(lens)]) for p in (c.k_pool, c.v_pool))
    pre = g.gqa_prefill_attn(c.q, k, v, _i32(c.starts), c.scale)
    assert float((out.double() - pre.double()).abs().max()) <= 2.0 ** -5
    c = Case([1, 1, 1], [130, 64, 500], Hq, Hkv, D, bs, seed=9, pad=0, wide=False)
    out = c.check()
    dec = g.gqa_decode_attn_paged(c.q, c.k_pool, c.v_pool, c.args[3], c.args[4], c.scale)
    assert float((out.double() - dec.double()).abs().max()) <= 2.0 ** -6


def test_bad_bounds_lengths_and_entries_are_reported_and_the_others_served():
    c = Case([4, 40, 9, 3], [100, 50, 200, 30], 8, 2, 128, 16, seed=10)
    before = torch.full((c.q.shape[0], 8, 128), 7.25, dtype=torch.bfloat16, device="cuda")
    ref, mag = c.ref()
    q, k, v, table, kv, cu, scale = c.args

    def others(out, a, e):  # (another call divides the work otherwise: within the tolerance, not to the bit)
        r = ref.clone()
        r[a:e] = NAN
        c.check(torch.cat([out[:a], before[a:e], out[e:]]), before, (r, mag))

    # a length outside the table row: zeros
    for bad in (-1, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        kv2 = kv.clone()
        kv2[1] = bad
        for f in (g.gqa_extend_attn, g.gqa_cross_attn):
            out = f(q, k, v, table, kv2, cu, scale, out=before.clone())
            _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
            assert not bool(out[4:44].any())
            if f is g.gqa_extend_attn:
                others(out, 4, 44)
    # bounds that are none, of sequences 1 and 2: skipped
    cu2 = cu.clone()
    cu2[2] = q.shape[0] + 1
    out = g.gqa_extend_attn(q, k, v, table, kv, cu2, scale, out=before.clone())
    _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
    others(out, 4, 53)
    assert bool((out[4:53] == 7.25).all())
    # entries: a block of zeros
    for bad in (-1, k.shape[0], 2 ** 31 - 1):
        t2 = table.clone()
        t2[2, 3] = bad
        out = g.gqa_extend_attn(q, k, v, t2, kv, cu, scale, out=before.clone())
        _raises(g.KVATTN_ERR_DEVICE_BOUNDS)
        k2, v2 = k.clone(), v.clone()
        k2[table[2, 3]] = 0
        v2[table[2, 3]] = 0
        want = g.gqa_extend_attn(q, k2, v2, table, kv, cu, scale, out=before.clone())
        g.check_device_error()
        assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_reports_and_the_next_call_is_clean(D):
    for c in (Case([200, 1], [700, 900], 8, 2, D, 64, seed=11), Case([1] * 9, [700, 900, 5] * 3, 8, 2, D, 64, seed=12)):
        g.set_wait_limit(1)
        try:
            c.run()
            _raises(g.KVATTN_ERR_TIMEOUT)
        finally:
            g.set_wait_limit(0)
        c.check()


def test_graphs_side_by_side_other_streams_and_release():
    cases = [Case([1] * 8, [3000 + 7 * i] * 8, 64, 8, 128, 64, seed=20 + i) for i in range(3)]
    refs = [c.ref() for c in cases]
    outs = [torch.zeros_like(c.q) for c in cases]
    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            c.run(out=o.contiguous() if not o.is_contiguous() else o)
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    g.check_device_error()
    for c, o, r in zip(cases, outs, refs):
        c.check(o, ref=r)
    # eager calls on streams of their own, beside each other
    got = []
    for _ in range(5):
        got = [c.run(stream=st) for c, st in zip(cases, streams)]
    torch.cuda.synchronize()
    for c, o, r in zip(cases, got, refs):
        c.check(o, ref=r)
    del graphs, gr
    g.release()
    cases[0].check(ref=refs[0])


def test_calls_back_to_back_with_the_rows_written_before_each():
    # append, attend, append, attend: each call sees the rows of the append before it
    Hq, Hkv, D, bs, B = 8, 2, 128, 16, 6
    nblk, maxb = B * 20, 20
    table = torch.randperm(nblk, generator=_gen(1), device="cuda", dtype=torch.int32).view(B, maxb)
    pools = [torch.full((nblk, Hkv, bs, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cos = torch.ones(400, D // 2, device="cuda")
    sin = torch.zeros(400, D // 2, device="cuda")
    hist = [[], []]
    outs = []
    for step, n in enumerate([37, 1, 1, 50, 1, 3, 1, 1]):
        qkv = _normal((B * n, Hq + 2 * Hkv, D), step)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = (lens[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)[None, :]).flatten()
        b = torch.arange(B, device="cuda").repeat_interleave(n)
        slots = table[b, (pos // bs).long()].long() * bs + pos % bs
        g.kv_append_rope(q, k, v, pos, cos, sin, slots, *pools, q_out=q)
        lens = lens + n
        cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
        outs.append((q, g.gqa_extend_attn(q, *pools, table, lens, cu, 0.09), n))
        for h, x in zip(hist, (k, v)):
            h.append(x.reshape(B, n, Hkv, D))
    g.check_device_error()
    K, V = (torch.cat(h, 1).double().repeat_interleave(Hq // Hkv, 2) for h in hist)
    at = 0
    for q, out, n in outs:
        e = at + n
        s = torch.einsum("bihd,bjhd->bhij", q.view(B, n, Hq, D).double(), K[:, :e]) * 0.09
        i = torch.arange(at, e, device="cuda")[:, None]
        s = s.masked_fill(torch.arange(e, device="cuda")[None, :] > i, -math.inf)
        w = torch.softmax(s, 3)
        ref = torch.einsum("bhij,bjhd->bihd", w, V[:, :e])
        mag = torch.einsum("bhij,bjhd->bihd", w, V[:, :e].abs())
        o = out.view(B, n, Hq, D).double()
        assert float(((o - ref).abs() - (2.0 ** -8 + 2.0 ** -10) * mag - 2.0 ** -8 * o.abs()).max()) <= 0
        at = e


def test_past_32_bits():
    # pools of 2.6e9 values each, the sequence's blocks at both ends
    Hq, Hkv, D, bs = 8, 8, 128, 128
    nblk = 20_000
    pools = [torch.zeros((nblk, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids = [nblk - 1, 0, nblk - 2, 16_384, 16_383]
    small = [_normal((len(ids), Hkv, bs, D), i) for i in range(2)]
    for p, s in zip(pools, small):
        p[torch.tensor(ids, device="cuda")] = s
    q = _normal((30, Hq, D), 5)
    cu, kv = _i32([0, 30]), _i32([5 * bs - 3])
    got = g.gqa_extend_attn(q, *pools, _i32([ids]), kv, cu, 0.1)
    want = g.gqa_extend_attn(q, *small, _i32([range(5)]), kv, cu, 0.1)
    g.check_device_error()
    assert torch.equal(got, want)
    del pools
    # 300 000 packed rows of 64 heads of 128: 2.5e9 values of q and out
    N = 300_000
    q = torch.zeros((N, 64, D), dtype=torch.bfloat16, device="cuda")
    rows = _normal((100, 64, D), 6)
    q[N - 100:] = rows
    got = g.gqa_cross_attn(q, *small, _i32([range(5), range(5)]), _i32([200, 600]), _i32([0, N - 100, N]), 0.1)
    want = g.gqa_cross_attn(rows, *small, _i32([range(5)]), _i32([600]), _i32([0, 100]), 0.1)
    g.check_device_error()
    over = (got[N - 100:].double() - want.double()).abs()
    assert float(over.max()) <= 2.0 ** -6  # (another division into pieces)
    mean = small[1].permute(0, 2, 1, 3).reshape(-1, Hkv, D)[:200].double().mean(0).repeat_interleave(8, 0)
    assert float((got[N // 2].double() - mean).abs().max()) <= 2.0 ** -8
