"""Attention over 8-bit caches where one position's weight stands far above
thousands of others that together hold much of the output (an attention sink
before a long cache), against the definition in 64 bits over the dequantized
cache.

The bound.  A weight times its value scale is rounded to binary16 (2^-11) and
enters the product as three E4M3 parts in units of 1, 2^-5 and 2^-10, which
lose at most half of the last part's smallest step, 2^-20, where the largest
value scale stands at 32 or more: 2^-25 of that scale times |code|, per
position, over a sum of weights of at least 1.  q enters as E4M3 parts, off by
at most 2^-17 of its head's largest |q|, and scores of D products in fp32 add
D 2^-24 sum|q k|: both move weights and their sum.  A sum over n positions is
taken in n / 32 steps of the tensor core (2^-23 of it each, n 2^-28) and n / 128
additions (less).  Last the output's own rounding: 2^-8 for bf16 (paged), 2^-20
for fp32 (division and the join of the three parts).
"""
import math

import numpy as np
import pytest
import torch

import grouped_query_kv_gb300 as g

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_query_kv_gb300 import build
    build.build()
    g.set_tuning(0, 0)
    yield
    g.set_tuning(0, 0)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make(lens, gaps, Hq, Hkv, D, sigma, seed):
    """q [B, Hq, D] and bf16 K/V rows of each request: request b's position
    at[b] scores gaps[b] above the others' mean for every head, the others
    N(0, sigma) about it; values of mean 0.7, the high one's near zero."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    q = normal(len(lens), Hq, D)
    q[:, :, 0] = 8.0
    rows = []
    for b, (n, gap) in enumerate(zip(lens, gaps)):
        k = normal(n, Hkv, D) * sigma
        v = normal(n, Hkv, D) + 0.7
        k[:, :, 0] = 0
        at = (0, n - 1, n // 2)[b % 3]
        k[at] = 0
        k[at, :, 0] = gap * math.sqrt(D) / 8.0
        v[at] = 0.01
        rows.append((k.to(torch.bfloat16), v.to(torch.bfloat16)))
    return q.to(torch.bfloat16), rows


def check(out, q, kvs, scale, half_ulp):
    """kvs: per request (k, v, |codes| of v, value scales [n, Hkv]) in 64 bits."""
    B, Hq, D = q.shape
    for b, (k, v, code, vs) in enumerate(kvs):
        n, Hkv = k.shape[:2]
        for h in range(Hkv):
            qs = q[b].double()[h * (Hq // Hkv):(h + 1) * (Hq // Hkv)]
            s = qs @ k[:, h].T * scale
            w = torch.exp(s - s.amax(1, keepdim=True))
            total = w.sum(1, keepdim=True)
            w = w / total
            ref, mag = w @ v[:, h], w @ v[:, h].abs()
            ds = scale * (2.0 ** -17 * qs.abs().amax(1, keepdim=True) * k[:, h].abs().sum(1).max()
                          + D * 2.0 ** -24 * (qs.abs() @ k[:, h].abs().T).amax(1, keepdim=True))
            lost = 2.0 ** -25 * vs[:, h].max() * code[:, h].sum(0) / total
            err = (2.0 ** -11 + 2 * ds + n * 2.0 ** -28) * mag + lost
            o = out[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
            over = (o - ref).abs() - err - half_ulp * (ref.abs() + err)
            assert bool(torch.isfinite(o).all()) and float(over.max()) <= 0, (b, h, float(over.max()))


CASES = [([8192, 20001, 32768, 9000, 8192], [9, 10, 11, 12, 13], 1.0),
         ([32768, 32768, 8192], [12, 15, 11], 0.5)]
HEADS = [(128, 8, 2), (128, 24, 1), (128, 48, 1), (128, 64, 1), (256, 16, 1), (256, 32, 1), (256, 48, 1)]


@pytest.mark.parametrize("lens,gaps,sigma", CASES, ids=["sigma1", "sigma05"])
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("ctas", [0, 1])  # split segments, and whole ones
def test_paged_8_bit(D, Hq, Hkv, lens, gaps, sigma, ctas):
    bs = 64
    q, rows = make(lens, gaps, Hq, Hkv, D, sigma, seed=D + Hq)
    blocks = [-(-n // bs) for n in lens]
    nblk = sum(blocks)
    ids = np.random.default_rng(D).permutation(nblk)
    table = np.full((len(lens), max(blocks)), -1, np.int32)
    for b, n in enumerate(blocks):
        table[b, :n] = ids[sum(blocks[:b]):sum(blocks[:b]) + n]
    codes = [torch.zeros((nblk, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((nblk, Hkv), device="cuda") for _ in range(2)]
    g.kv_append_paged_fp8(*codes, *scales, torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]),
                          _i32(table), _i32([0] * len(lens)), _i32(np.concatenate([[0], np.cumsum(lens)])))
    scale = 1 / math.sqrt(D)
    g.set_tuning(0, ctas)
    try:
        out = g.gqa_decode_attn_paged_fp8(q, *codes, *scales, _i32(table), _i32(lens), scale)
        g.check_device_error()
    finally:
        g.set_tuning(0, 0)
    kvs = []
    for b, n in enumerate(lens):
        at = torch.as_tensor(table[b, :blocks[b]].astype(np.int64), device="cuda")
        c = [x[at].view(torch.float8_e4m3fn).double().transpose(1, 2).reshape(-1, Hkv, D)[:n] for x in codes]
        s = [x[at].double().repeat_interleave(bs, 0)[:n] for x in scales]
        kvs.append((c[0] * s[0][:, :, None], c[1] * s[1][:, :, None], c[1].abs(), s[1]))
    check(out, q, kvs, scale, 2.0 ** -8)


@pytest.mark.parametrize("lens,gaps,sigma", CASES, ids=["sigma1", "sigma05"])
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("ctas", [0, 1])
def test_contiguous_8_bit(D, Hq, Hkv, lens, gaps, sigma, ctas):
    q, rows = make(lens, gaps, Hq, Hkv, D, sigma, seed=D + Hq + 1)
    cache = [torch.zeros((len(lens), Hkv, max(lens), D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, n in enumerate(lens):
        for c, r in zip(cache, rows[b]):
            c[b, :, :n] = r.transpose(0, 1)
    (kc, ks), (vc, vs) = (g.kv_quantize_fp8(c) for c in cache)
    scale = 1 / math.sqrt(D)
    g.set_tuning(0, ctas)
    try:
        out = g.gqa_decode_attn_fp8(q, kc, vc, ks, vs, _i32(lens), scale)
        g.check_device_error()
    finally:
        g.set_tuning(0, 0)
    kvs = []
    for b, n in enumerate(lens):
        c = [x[b, :, :n].view(torch.float8_e4m3fn).double().transpose(0, 1) for x in (kc, vc)]
        s = [x[b, :, :n].double().T for x in (ks, vs)]
        kvs.append((c[0] * s[0][:, :, None], c[1] * s[1][:, :, None], c[1].abs(), s[1]))
    check(out, q, kvs, scale, 2.0 ** -20)


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("paged", [False, True])
def test_a_query_entry_far_above_the_others(D, Hq, Hkv, paged):
    """One entry of q stands 2^11 to 2^12 above the others, where K is zero: the
    scores come from the others, which the parts hold exactly (2^14 below the
    largest they still do).  So what moves a score is the sum in fp32 alone."""
    lens, bs, scale = [1, 5, 40, 200, 1000], 64, 0.5
    gen = torch.Generator(device="cuda").manual_seed(D + Hq)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    q = (0.5 + 0.5 * uniform(len(lens), Hq, D)) * (2 * (uniform(len(lens), Hq, D) < 0.5) - 1)
    q[:, :, 3] = 2048.0
    q = q.to(torch.bfloat16)
    cache = [torch.randn((len(lens), Hkv, 1024, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    cache[0][:, :, :, 3] = 0
    if paged:
        table = _i32(np.arange(len(lens) * 16).reshape(len(lens), 16))
        codes = [torch.zeros((len(lens) * 16, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros((len(lens) * 16, Hkv), device="cuda") for _ in range(2)]
        rows = [c.transpose(1, 2).reshape(-1, Hkv, D).contiguous() for c in cache]
        g.kv_append_paged_fp8(*codes, *scales, *rows, table, _i32([0] * len(lens)),
                              _i32(np.arange(len(lens) + 1) * 1024))
        out = g.gqa_decode_attn_paged_fp8(q, *codes, *scales, table, _i32(lens), scale)
        codes = [c.view(len(lens), 16, Hkv, bs, D).transpose(2, 3).reshape(-1, 1024, Hkv, D) for c in codes]
        scales = [x.view(len(lens), 16, Hkv).repeat_interleave(bs, 1) for x in scales]
    else:
        (kc, ks), (vc, vs) = (g.kv_quantize_fp8(c) for c in cache)
        out = g.gqa_decode_attn_fp8(q, kc, vc, ks, vs, _i32(lens), scale)
        codes = [c.transpose(1, 2) for c in (kc, vc)]
        scales = [x.transpose(1, 2) for x in (ks, vs)]
    g.check_device_error()
    for b, n in enumerate(lens):
        k, v = (c[b, :n].contiguous().view(torch.float8_e4m3fn).double() * x[b, :n, :, None].double()
                for c, x in zip(codes, scales))
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            qs = q[b, heads].double()
            w = torch.softmax(qs @ k[:, h].T * scale, 1)
            ref, mag = w @ v[:, h], w @ v[:, h].abs()
            ds = scale * D * 2.0 ** -24 * (qs.abs() @ k[:, h].abs().T).amax(1, keepdim=True)
            lost = 2.0 ** -25 * v[:, h].abs().max() * n
            err = (2.0 ** -11 + 2 * ds + 2.0 ** -18) * mag + lost
            o = out[b, heads].double()
            over = (o - ref).abs() - err - (2.0 ** -8 if paged else 2.0 ** -20) * (ref.abs() + err)
            assert float(over.max()) <= 0, (b, h, float(over.max()))


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("small", [2.0 ** -9, 2.0 ** -30, 2.0 ** -110])
@pytest.mark.parametrize("ctas", [0, 1])
def test_value_scales_of_zero_before_others(D, Hq, Hkv, small, ctas):
    """The first tiles' value scales are 0 (of whole blocks, paged, and of rows),
    so they say nothing about the unit that the others need."""
    lens, zeros, bs, L = [1000, 128, 300, 129], [300, 0, 256, 128], 32, 1024
    gen = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn((len(lens), Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    codes = [torch.randint(0, 120, (len(lens) * L // bs, Hkv, bs, D), generator=gen, device="cuda", dtype=torch.uint8)
             for _ in range(2)]
    nb, scale = L // bs, 1 / math.sqrt(D)
    ks = torch.full((len(lens) * nb, Hkv), 2.0 ** -7, device="cuda")
    vs = torch.full((len(lens) * nb, Hkv), small, device="cuda")
    for b, z in enumerate(zeros):
        vs[b * nb:b * nb + z // bs] = 0
    table = _i32(np.arange(len(lens) * nb).reshape(len(lens), nb))
    cont = [c.view(len(lens), nb, Hkv, bs, D).permute(0, 2, 1, 3, 4).reshape(len(lens), Hkv, L, D).contiguous()
            for c in codes]
    rows = [x.view(len(lens), nb, Hkv).permute(0, 2, 1).repeat_interleave(bs, 2).contiguous() for x in (ks, vs)]
    g.set_tuning(0, ctas)
    try:
        out = g.gqa_decode_attn_paged_fp8(q, *codes, ks, vs, table, _i32(lens), scale)
        out32 = g.gqa_decode_attn_fp8(q, *cont, *rows, _i32(lens), scale)
        g.check_device_error()
    finally:
        g.set_tuning(0, 0)
    kvs = []
    for b, n in enumerate(lens):
        c = [x[b, :, :n].contiguous().view(torch.float8_e4m3fn).double().transpose(0, 1) for x in cont]
        s = [x[b, :, :n].double().T for x in rows]
        kvs.append((c[0] * s[0][:, :, None], c[1] * s[1][:, :, None], c[1].abs(), s[1]))
    check(out, q, kvs, scale, 2.0 ** -8)
    check(out32, q, kvs, scale, 2.0 ** -20)
