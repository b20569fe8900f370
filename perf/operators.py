"""Measured cases of the operators that take prompts into a paged KV cache.

A request reaches the cache in this order: blocks and slots for its tokens
(kv_block_tables), its K/V rows written there (kv_append_slots into a bf16
pool, kv_append_paged_fp8 into an 8-bit pool with one scale per block and K/V
head), its prompt's own attention (gqa_prefill_attn), and single-token steps
over the 8-bit pool (gqa_decode_attn_paged_fp8).

`run` computes each operator in plain torch operations where `own` is false and
calls the library where it is true; `exact` gives the same outputs from the
definitions in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 running requests: a block for the few that cross a block boundary
        dict(name="tables_step64", op="tables", B=64, new_max=1, new_min=1, cached_max=8191, bs=16, pad=0),
        # admission of a large batch of prompts of ragged lengths, some requests idle
        dict(name="tables_prompts1024", op="tables", B=1024, new_max=2047, new_min=0, cached_max=4096, bs=16,
             pad=37),
        # one decode step's rows of 64 requests, 8 K/V heads of 128
        dict(name="slots_step64", op="slots", N=64, Hq=64, Hkv=8, D=128, bs=16, pad=3),
        # the rows of a packed batch of prompts, sliced out of one fused projection
        dict(name="slots_prompts64k", op="slots", N=65536, Hq=8, Hkv=8, D=128, bs=64, pad=0),
        # a chat turn: a few short prompts (latency), 64 heads over 8 K/V heads of 128
        dict(name="prefill_short", op="prefill", B=4, len_min=1, len_max=97, Hq=64, Hkv=8, D=128, window=0, pad=5),
        # one long prompt at the same head layout: the largest amount of work
        dict(name="prefill_8192", op="prefill", B=1, len_min=8192, len_max=8192, Hq=64, Hkv=8, D=128, window=0,
             pad=0),
        # several prompts of ragged lengths, multi-query heads of 256
        dict(name="prefill_mqa256", op="prefill", B=8, len_min=0, len_max=4095, Hq=16, Hkv=1, D=256, window=0,
             pad=11),
        # a local attention layer, one head per K/V head, heads of 64
        dict(name="prefill_local64", op="prefill", B=3, len_min=1000, len_max=6001, Hq=16, Hkv=16, D=64,
             window=1024, pad=0),
        # one decode step's rows into the 8-bit pool, most of them into blocks partly filled
        dict(name="fp8_step64", op="append8", B=64, new_min=1, new_max=1, cached_max=1000, Hq=64, Hkv=8, D=128,
             bs=16, pad=0),
        # a packed batch of ragged prompts into the 8-bit pool
        dict(name="fp8_prompts32", op="append8", B=32, new_min=0, new_max=4095, cached_max=100, Hq=8, Hkv=8, D=128,
             bs=64, pad=9),
        # a few short requests over the 8-bit pool (latency)
        dict(name="attn8_short", op="attn8", B=5, len_min=0, len_max=301, Hq=32, Hkv=8, D=128, bs=32),
        # 32 ragged requests up to 8192 tokens, 64 heads over 8 K/V heads of 128, 16-position blocks
        dict(name="attn8_ragged8192", op="attn8", B=32, len_min=1, len_max=8192, Hq=64, Hkv=8, D=128, bs=16),
    ]


def _log_int(rng, lo, hi):
    """An int in [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "slots", "prefill", "append8", "attn8"])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    bs = rng.choice([16, 32, 64, 128])
    if op == "tables":
        B = _log_int(rng, 1, 1024)
        new_max = _log_int(rng, 1, 2047)
        return dict(op=op, B=B, new_min=rng.choice([0, 1]) if B > 4 else 1, new_max=new_max,
                    cached_max=_log_int(rng, 1, 4096), bs=bs, pad=pad)
    if op == "slots":
        N = _log_int(rng, 1, max(1, 65536 * 8 * 128 // (Hkv * D) // 2))
        N = min(N, 65536)
        return dict(op=op, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, pad=min(pad, N - 1))
    if op == "prefill":
        B = _log_int(rng, 1, 16)
        Hq = Hkv * G
        most = int(math.sqrt(64 * 8192 * 8192 * 128 / (B * Hq * D)))  # the long prompt's work
        top = _log_int(rng, 1, min(8191, most))
        window = rng.choice([0, 0, _log_int(rng, 1, top)])
        least = rng.choice([0 if B > 4 else 1, 1, max(1, top // 2)])
        return dict(op=op, B=B, len_min=least, len_max=top, Hq=Hq, Hkv=Hkv, D=D, window=window, pad=pad)
    if op == "append8":
        B = _log_int(rng, 1, 64)
        least = rng.choice([0, 1]) if B > 4 else 1
        new_max = _log_int(rng, 1, max(1, min(4095, 32 * 4095 * 8 * 128 // (B * Hkv * D))))
        return dict(op=op, B=B, new_min=least, new_max=new_max, cached_max=_log_int(rng, 1, 1000), Hq=Hkv * G,
                    Hkv=Hkv, D=D, bs=bs, pad=pad)
    D = rng.choice([128, 256])
    B = _log_int(rng, 1, 32)
    top = _log_int(rng, 1, min(32768, 32 * 8192 * 8 * 128 // (B * Hkv * D)))
    least = rng.choice([0 if B > 4 else 1, 1, max(1, top // 2)])
    return dict(op=op, B=B, len_min=least, len_max=top, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs)


# ------------------------------------------------------------------ inputs

def _host_ints(seed, salt, lo, hi, n):
    g = torch.Generator().manual_seed(seed * 1000003 + salt)
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _starts(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)])


def _tables(seed, lens, bs, spare):
    """A block table in the order an allocator hands blocks out, and the pool's size: entries past a request's
    blocks are -1."""
    nb = (lens + bs - 1) // bs
    maxb = max(1, int(nb.max()))
    total = int(nb.sum()) + spare
    g = torch.Generator().manual_seed(seed * 1000003 + 5)
    phys = torch.randperm(total, generator=g)
    table = torch.full((len(lens), maxb), -1, dtype=torch.int64)
    used = torch.arange(maxb)[None, :] < nb[:, None]
    table[used] = phys[:int(nb.sum())]
    return table, phys[int(nb.sum()):], total


def _lens(case, seed):
    """The host's lengths of a case: (cached, new) of a writing case, (None, lens) of an attention. A case has one
    set of lengths, so that its outputs' shapes are its own; the seed gives their order."""
    B = case["B"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed * 1000003 + 4))
    if case["op"] in ("tables", "append8"):
        return (_host_ints(1, 1, 0, case["cached_max"], B)[order],
                _host_ints(1, 2, case["new_min"], case["new_max"], B)[order])
    return None, _host_ints(1, 3, case["len_min"], case["len_max"], B)[order]


def _pow2_scale(amax):
    """The smallest power of two s, 2^-100 at least, with amax <= 448 s."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes_pool(nblk, Hkv, bs, D, gen):
    """An 8-bit pool: codes of normal values and one scale per block and K/V head."""
    x = torch.randn((nblk, Hkv, bs, D), generator=gen, device="cuda")
    scale = _pow2_scale(x.abs().amax(dim=(2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    op = case["op"]
    gen = _gen(seed)
    st = dict(case)
    dev = "cuda"
    if op == "tables":
        cached, new = _lens(case, seed)
        bs = case["bs"]
        lens = cached + new
        table, _, _ = _tables(seed, cached, bs, 0)
        maxb = max(1, int(((lens + bs - 1) // bs).max()))
        wide = torch.full((case["B"], maxb), -1, dtype=torch.int64)
        n = min(maxb, table.shape[1])
        wide[:, :n] = table[:, :n]
        used = int((table >= 0).sum())
        need = int(((lens + bs - 1) // bs - (cached + bs - 1) // bs).sum())
        g = torch.Generator().manual_seed(seed * 1000003 + 6)
        free = torch.randperm(need + 64, generator=g) + used
        st.update(cached=cached.to(dev, torch.int32), new=new.to(dev, torch.int32), table=wide.to(dev, torch.int32),
                  free=free.to(dev, torch.int32),
                  free_count=torch.tensor([need + 64 - 7], dtype=torch.int32, device=dev),
                  free_out=torch.zeros(1, dtype=torch.int32, device=dev),
                  num_slots=int(new.sum()) + case["pad"])
        st["num_slots"] = max(1, st["num_slots"])
        return st
    if op == "slots":
        N, Hq, Hkv, D, bs = (case[k] for k in ("N", "Hq", "Hkv", "D", "bs"))
        qkv = _normal((N, Hq + 2 * Hkv, D), gen)
        nblk = (N + bs - 1) // bs + 4
        g = torch.Generator().manual_seed(seed * 1000003 + 7)
        # whole blocks in an allocator's order, rows in order within a block
        first = torch.randperm(nblk, generator=g)[:(N + bs - 1) // bs] * bs
        slots = (first[:, None] + torch.arange(bs)[None, :]).reshape(-1)[:N].clone()
        used = N - case["pad"]
        slots[used:] = -1
        pool = torch.zeros((2, nblk, Hkv, bs, D), dtype=torch.bfloat16, device=dev)
        st.update(k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], slots=slots.to(dev), used=used, k_pool=pool[0],
                  v_pool=pool[1])
        return st
    if op == "prefill":
        _, lens = _lens(case, seed)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        total = int(lens.sum())
        N = max(1, total + case["pad"])
        qkv = _normal((N, Hq + 2 * Hkv, D), gen)
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:],
                  cu=_starts(lens).to(dev, torch.int32), longest=max(1, int(lens.max())),
                  scale=1.0 / math.sqrt(D), out=torch.zeros((N, Hq, D), dtype=torch.bfloat16, device=dev))
        return st
    if op == "append8":
        cached, new = _lens(case, seed)
        Hq, Hkv, D, bs = (case[k] for k in ("Hq", "Hkv", "D", "bs"))
        table, _, nblk = _tables(seed, cached + new, bs, 3)
        N = max(1, int(new.sum()) + case["pad"])
        kc, ks = _codes_pool(nblk, Hkv, bs, D, gen)
        vc, vs = _codes_pool(nblk, Hkv, bs, D, gen)
        qkv = _normal((N, Hq + 2 * Hkv, D), gen)
        # keys of some tokens stand out, so that a block's scale may have to grow
        tall = (torch.rand((N, 1, 1), generator=gen, device=dev) < 0.2)
        qkv = torch.where(tall, qkv * 4, qkv)
        st.update(k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], kc=kc, vc=vc, ks=ks, vs=vs,
                  table=table.to(dev, torch.int32), cached=cached.to(dev, torch.int32),
                  cu=_starts(new).to(dev, torch.int32), total=int(new.sum()))
        return st
    _, lens = _lens(case, seed)
    Hq, Hkv, D, bs = (case[k] for k in ("Hq", "Hkv", "D", "bs"))
    table, _, nblk = _tables(seed, lens, bs, 2)
    kc, ks = _codes_pool(nblk, Hkv, bs, D, gen)
    vc, vs = _codes_pool(nblk, Hkv, bs, D, gen)
    st.update(q=_normal((case["B"], Hq, D), gen), kc=kc, vc=vc, ks=ks, vs=vs, table=table.to(dev, torch.int32),
              lens=lens.to(dev, torch.int32), scale=1.0 / math.sqrt(D),
              out=torch.zeros((case["B"], Hq, D), dtype=torch.bfloat16, device=dev))
    return st


# ------------------------------------------------------------- plain forms

def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_tables(s):
    bs = s["bs"]
    cached, new = s["cached"].long(), s["new"].long()
    have = (cached + bs - 1) // bs
    upto = (cached + new + bs - 1) // bs
    need = upto - have
    before = need.cumsum(0) - need
    k = torch.arange(s["table"].shape[1], device=cached.device)[None, :]
    fresh = (k >= have[:, None]) & (k < upto[:, None])
    at = s["free_count"].long() - 1 - (before[:, None] + k - have[:, None])
    taken = s["free"].long()[at.clamp(0, s["free"].shape[0] - 1)]
    table = torch.where(fresh, taken, s["table"].long())
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(s["num_slots"], device=cached.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=cached.shape[0] - 1)
    pos = cached[b] + t - cu[b]
    slot = table[b, (pos // bs).clamp(max=table.shape[1] - 1)] * bs + pos % bs
    slots = torch.where(t < cu[-1], slot, torch.full_like(slot, -1))
    left = (s["free_count"].long() - need.sum()).to(torch.int32)
    return table.to(torch.int32), cu.to(torch.int32), slots, left


def _plain_slots(s):
    n, bs = s["used"], s["bs"]
    at = s["slots"][:n]
    s["k_pool"][at // bs, :, at % bs] = s["k"][:n]
    s["v_pool"][at // bs, :, at % bs] = s["v"][:n]
    return s["k_pool"], s["v_pool"]


def _plain_prefill(s):
    Hq, Hkv, D, L = s["Hq"], s["Hkv"], s["D"], s["longest"]
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    B, N = lens.shape[0], s["q"].shape[0]
    i = torch.arange(L, device=cu.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=N - 1)
    real = i[None, :] < lens[:, None]                                         # [B, L]
    q = s["q"].float()[rows].view(B, L, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    k = s["k"].float()[rows].permute(0, 2, 3, 1)                              # [B, Hkv, D, L]
    v = torch.where(real[:, None, :, None], s["v"].float()[rows].permute(0, 2, 1, 3), 0.0)
    p = torch.matmul(q, k).view(B, Hkv, Hq // Hkv, L, L)
    p *= s["scale"]
    seen = i[None, :] <= i[:, None]
    if s["window"]:
        seen = seen & (i[None, :] > i[:, None] - s["window"])
    p.masked_fill_(~seen, -math.inf)
    p -= p.amax(dim=-1, keepdim=True)
    p.exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, L), v).view(B, Hkv, Hq // Hkv, L, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B * L, Hq, D).to(torch.bfloat16)
    t = torch.arange(N, device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    mine = o[(b * L + t - cu[b]).clamp(0, B * L - 1)]
    return torch.where((t < cu[-1])[:, None, None], mine, s["out"])


def _plain_write8(codes, scale, x, blk, row, first_blk, first_rows, bs):
    amax = x.abs().amax(dim=-1)                                               # [N, Hkv]
    most = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand_as(amax), amax, "amax")
    written = torch.zeros(scale.shape[0], dtype=torch.int64, device=x.device).index_fill_(0, blk, 1) > 0
    kept = torch.zeros_like(written, dtype=torch.int64).scatter_reduce_(0, first_blk, first_rows, "amax")
    fresh = _pow2_scale(most)
    grown = torch.where((kept > 0)[:, None], torch.maximum(scale, fresh), fresh)
    now = torch.where(written[:, None], grown, scale)
    again = (_values(codes) * (scale / now)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    old = torch.arange(bs, device=x.device)[None, :] < kept[:, None]          # rows that were there
    codes.copy_(torch.where(old[:, None, :, None], again, codes))
    codes[blk, :, row] = (x / now[blk][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(now)
    return codes.view(torch.float8_e4m3fn), scale


def _plain_append8(s):
    bs, n = s["bs"], s["total"]
    cu, cached, table = s["cu"].long(), s["cached"].long(), s["table"].long()
    t = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = cached[b] + t - cu[b]
    blk, row = table[b, pos // bs], pos % bs
    # the rows already in the block that a request's first new token goes to
    some = cu[1:] > cu[:-1]
    first_blk = table.gather(1, (cached // bs).clamp(max=table.shape[1] - 1)[:, None])[:, 0].clamp(min=0)
    first_rows = torch.where(some, cached % bs, torch.zeros_like(cached))
    kc, ks = _plain_write8(s["kc"], s["ks"], s["k"][:n].float(), blk, row, first_blk, first_rows, bs)
    vc, vs = _plain_write8(s["vc"], s["vs"], s["v"][:n].float(), blk, row, first_blk, first_rows, bs)
    return kc, ks, vc, vs


def _plain_attn8(s):
    B, Hq, D = s["q"].shape
    Hkv, bs = s["Hkv"], s["bs"]
    at = s["table"].long().clamp(min=0)
    L = at.shape[1] * bs
    k = (_values(s["kc"][at]) * s["ks"][at][..., None, None]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    v = (_values(s["vc"][at]) * s["vs"][at][..., None, None]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    seen = torch.arange(L, device=at.device)[None, :] < s["lens"].long()[:, None]
    v = torch.where(seen[:, None, :, None], v, 0.0)
    p = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, D), k.transpose(2, 3)) * s["scale"]
    p = torch.where(seen[:, None, None, :], p, -math.inf)
    top = p.amax(dim=-1, keepdim=True)
    p = torch.exp(p - torch.where(top == -math.inf, 0.0, top))
    o = torch.matmul(p, v) / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    return o.view(B, Hq, D).to(torch.bfloat16)


_PLAIN = dict(tables=_plain_tables, slots=_plain_slots, prefill=_plain_prefill, append8=_plain_append8,
              attn8=_plain_attn8)


# ------------------------------------------------------- the library's calls

def _own_tables(g, s):
    cu, slots, left = g.kv_block_tables(s["cached"], s["new"], s["table"], s["free"], s["free_count"], s["bs"],
                                        s["num_slots"], free_count_out=s["free_out"])
    return s["table"], cu, slots, left


def _own_slots(g, s):
    g.kv_append_slots(s["k_pool"], s["v_pool"], s["k"], s["v"], s["slots"])
    return s["k_pool"], s["v_pool"]


def _own_prefill(g, s):
    return g.gqa_prefill_attn(s["q"], s["k"], s["v"], s["cu"], s["scale"], out=s["out"], window=s["window"] or None)


def _own_append8(g, s):
    g.kv_append_paged_fp8(s["kc"], s["vc"], s["ks"], s["vs"], s["k"], s["v"], s["table"], s["cached"], s["cu"])
    return s["kc"].view(torch.float8_e4m3fn), s["ks"], s["vc"].view(torch.float8_e4m3fn), s["vs"]


def _own_attn8(g, s):
    return g.gqa_decode_attn_paged_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"],
                                       out=s["out"])


_OWN = dict(tables=_own_tables, slots=_own_slots, prefill=_own_prefill, append8=_own_append8, attn8=_own_attn8)


def run(state):
    if own:
        import grouped_query_kv_gb300 as g
        return _OWN[state["op"]](g, state)
    return _PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and operations that one pass cannot do without: each input read once, each output written once."""
    op = case["op"]
    if op == "slots":
        row = case["Hkv"] * case["D"] * 2
        return dict(bytes=(case["N"] - case["pad"]) * 4 * row + case["N"] * 8, flops=0)
    if op == "prefill":
        _, lens = _lens(case, 1)
        Hq, Hkv, D, w = case["Hq"], case["Hkv"], case["D"], case["window"]
        rows = int(lens.sum())
        pairs = 0
        for n in lens.tolist():
            m = min(n, w) if w else n
            pairs += m * (m + 1) // 2 + (n - m) * m
        return dict(bytes=max(1, rows) * (2 * Hq + 2 * Hkv) * D * 2, flops=4 * pairs * Hq * D)
    if op == "attn8":
        _, lens = _lens(case, 1)
        bs, Hkv, D = case["bs"], case["Hkv"], case["D"]
        blocks = int(((lens + bs - 1) // bs).sum())
        rows = int(lens.sum())
        return dict(bytes=2 * rows * Hkv * D + blocks * (8 * Hkv + 4) + case["B"] * (case["Hq"] * D * 4 + 4),
                    flops=4 * rows * case["Hq"] * D)
    B, bs = case["B"], case["bs"]
    cached, new = _lens(case, 1)
    n = int(new.sum())
    fresh = int(((cached + new + bs - 1) // bs - (cached + bs - 1) // bs).sum())
    if op == "tables":
        return dict(bytes=B * 12 + fresh * 8 + (n + case["pad"]) * 8, flops=0)
    Hkv, D = case["Hkv"], case["D"]
    blocks = int(torch.where(new > 0, (cached + new + bs - 1) // bs - cached // bs, new).sum())
    return dict(bytes=2 * (n * Hkv * D * 3 + blocks * (Hkv * 4 + 4)) + B * 8, flops=0)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs of `run` from the definitions, request by request, in 64 bits."""
    def _exact_tables(s):
        bs = s["bs"]
        cached, new, free = s["cached"].tolist(), s["new"].tolist(), s["free"].tolist()
        table = s["table"].tolist()
        left, cu, slots = int(s["free_count"]), [0], []
        for b in range(len(cached)):
            for p in range(cached[b], cached[b] + new[b]):
                if p % bs == 0:
                    left -= 1
                    table[b][p // bs] = free[left]
                slots.append(table[b][p // bs] * bs + p % bs)
            cu.append(len(slots))
        slots += [-1] * (s["num_slots"] - len(slots))
        return (torch.tensor(table, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32),
                torch.tensor(slots, dtype=torch.int64), torch.tensor([left], dtype=torch.int32))

    def _exact_slots(s):
        out = []
        at = s["slots"][s["slots"] >= 0]
        for pool, rows in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])):
            nblk, Hkv, bs, D = pool.shape
            flat = pool.double().permute(0, 2, 1, 3).reshape(nblk * bs, Hkv, D)
            flat.index_copy_(0, at, rows[s["slots"] >= 0].double())
            out.append(flat.view(nblk, bs, Hkv, D).permute(0, 2, 1, 3))
        return tuple(out)

    def _exact_prefill(s):
        G = s["Hq"] // s["Hkv"]
        out = s["out"].double()
        cu = s["cu"].tolist()
        for a, e in zip(cu[:-1], cu[1:]):
            if a == e:
                continue
            j = torch.arange(e - a, device=out.device)
            far = j[:, None] - j[None, :]
            hidden = (far < 0) | (far >= s["window"]) if s["window"] else far < 0
            for h in range(s["Hq"]):
                x = (s["q"][a:e, h].double() @ s["k"][a:e, h // G].double().T) * s["scale"]
                x[hidden] = -math.inf
                out[a:e, h] = torch.softmax(x, dim=1) @ s["v"][a:e, h // G].double()
        return out

    def _exact_write8(codes, scale, x, s):
        """Rows of the pool as x / scale, unrounded."""
        bs = s["bs"]
        val, sc = codes.view(torch.float8_e4m3fn).double(), scale.clone()
        cu, cached, table = s["cu"].tolist(), s["cached"].tolist(), s["table"].tolist()
        for b in range(len(cached)):
            at, end = cu[b], cu[b + 1]
            while at < end:
                p = cached[b] + at - cu[b]
                blk, r = table[b][p // bs], p % bs
                n = min(bs - r, end - at)
                rows = x[at:at + n].double().permute(1, 0, 2)                     # [Hkv, n, D]
                e = torch.ceil(torch.log2(rows.abs().amax(dim=(1, 2)) / 448)).clamp(min=-100)
                now = torch.exp2(e)
                if r:
                    now = torch.maximum(now, sc[blk].double())
                    val[blk, :, :r] *= (sc[blk].double() / now)[:, None, None]
                val[blk, :, r:r + n] = rows / now[:, None, None]
                sc[blk] = now.float()
                at += n
        return val, sc.double()

    def _exact_append8(s):
        kc, ks = _exact_write8(s["kc"], s["ks"], s["k"], s)
        vc, vs = _exact_write8(s["vc"], s["vs"], s["v"], s)
        return kc, ks, vc, vs

    def _exact_attn8(s):
        B, Hq, D = s["q"].shape
        G, bs = Hq // s["Hkv"], s["bs"]
        out = torch.zeros((B, Hq, D), dtype=torch.float64, device=s["q"].device)
        for b, n in enumerate(s["lens"].tolist()):
            if not n:
                continue
            ids = s["table"][b, :(n + bs - 1) // bs].long()
            for h in range(s["Hkv"]):
                k = (s["kc"][ids, h].view(torch.float8_e4m3fn).double() * s["ks"][ids, h].double()[:, None, None])
                v = (s["vc"][ids, h].view(torch.float8_e4m3fn).double() * s["vs"][ids, h].double()[:, None, None])
                k, v = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
                x = s["q"][b, h * G:(h + 1) * G].double() @ k.T * s["scale"]
                out[b, h * G:(h + 1) * G] = torch.softmax(x, dim=1) @ v
        return out

    s = prepare(case, seed)
    return dict(tables=_exact_tables, slots=_exact_slots, prefill=_exact_prefill, append8=_exact_append8,
                attn8=_exact_attn8)[case["op"]](s)
