"""Measured cases of the operators around a paged KV cache that serve running requests.

A step normalises and rotates its tokens' queries and keys and writes their K/V rows to their slots (qk_norm_rope,
kv_append_rope); the tokens attend what their request has cached, themselves included (gqa_extend_attn), or an
encoder's states in the pool (gqa_cross_attn); requests are forked, their last block copied, and dropped
(kv_fork_blocks, kv_copy_blocks, kv_free_blocks), and the pool is compacted (kv_compact_blocks, kv_copy_blocks).

`run` computes each operator in plain torch operations where `own` is false and calls the library where it is true;
`exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 requests: 64 heads over 8 K/V heads of 128, rows to their slots
        dict(name="rope_step64", op="rope", N=64, Hq=64, Hkv=8, D=128, rd=128, pairs="half", norm=True, pool=True,
             max_pos=8192, bs=16, pad=3),
        # a packed batch of prompts at the same heads
        dict(name="rope_prompts16k", op="rope", N=16384, Hq=64, Hkv=8, D=128, rd=128, pairs="half", norm=True,
             pool=True, max_pos=32768, bs=64, pad=0),
        # multi-query heads of 256, half of the dims rotated in neighbouring pairs, packed keys out
        dict(name="rope_mqa256", op="rope", N=5001, Hq=16, Hkv=1, D=256, rd=128, pairs="next", norm=False, pool=False,
             max_pos=131072, bs=16, pad=9),
        # one decode step of 32 ragged requests over blocks of 16 positions
        dict(name="extend_step32", op="attn", causal=True, B=32, new_min=1, new_max=1, chunks=0, kv_min=1, kv_max=8191,
             Hq=64, Hkv=8, D=128, window=0, bs=16, pad=0),
        # a step of running requests, three of them taking 256 more tokens of their prompts
        dict(name="extend_mixed24", op="attn", causal=True, B=24, new_min=1, new_max=256, chunks=3, kv_min=1,
             kv_max=4095, Hq=32, Hkv=8, D=128, window=0, bs=32, pad=5),
        # four long prompts taken 2048 tokens at a time, 6144 cached: the largest amount of work
        dict(name="extend_chunk2048", op="attn", causal=True, B=4, new_min=2048, new_max=2048, chunks=0, kv_min=6144,
             kv_max=6144, Hq=64, Hkv=8, D=128, window=0, bs=64, pad=0),
        # multi-query heads of 256 on a local layer
        dict(name="extend_local256", op="attn", causal=True, B=8, new_min=0, new_max=511, chunks=0, kv_min=0,
             kv_max=4095, Hq=16, Hkv=1, D=256, window=1024, bs=64, pad=11),
        # one decode step of 64 requests over their encoder's states, one head per K/V head of 64
        dict(name="cross_step64", op="attn", causal=False, B=64, new_min=1, new_max=1, chunks=0, kv_min=1, kv_max=2048,
             Hq=16, Hkv=16, D=64, window=0, bs=64, pad=0),
        # the decoder's prompts over their encoder's states
        dict(name="cross_prompts16", op="attn", causal=False, B=16, new_min=1, new_max=255, chunks=0, kv_min=0,
             kv_max=2047, Hq=16, Hkv=16, D=64, window=0, bs=16, pad=7),
        # 64 of 256 requests forked (their last block copied) and the forks dropped
        dict(name="fork_step64", op="fork", R=256, n=64, kv_max=2047, Hkv=8, D=128, bs=16),
        # a pool of 65 536 blocks with every other one free, 1024 requests
        dict(name="compact_64k", op="compact", R=1024, per=32, shared=0.25, bs=16),
        # the blocks that a compaction moves, K and V
        dict(name="copy_8192", op="copy", n=8192, blocks=16384, Hkv=8, D=128, bs=16),
    ]


def _log_int(rng, lo, hi):
    """An int in [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "attn", "fork", "compact", "copy"])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    bs = rng.choice([16, 32, 64, 128])
    if op == "rope":
        N = _log_int(rng, 1, max(1, 16384 * 80 * 128 // (Hkv * (G + 2) * D)))
        N = min(N, 65536)
        return dict(op=op, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, rd=rng.choice([D, D, D // 2, 32]),
                    pairs=rng.choice(["half", "next"]), norm=rng.choice([True, False]), pool=rng.choice([True, False]),
                    max_pos=_log_int(rng, 16, 131072), bs=bs, pad=min(pad, N - 1))
    if op == "attn":
        B = _log_int(rng, 1, 64)
        Hq = Hkv * G
        causal = rng.choice([True, True, False])
        new_max = rng.choice([1, _log_int(rng, 1, 1024), _log_int(rng, 1, 2048)])
        most = 4 * 64 * 2048 * 8192 // (B * Hq * new_max)  # the long prompts' scores
        most = min(most * 128 // max(D, 128), 32 * 8192 * 8 * 128 // (B * Hkv * D))
        kv_max = _log_int(rng, 1, max(1, min(16383, most - new_max)))
        window = rng.choice([0, 0, _log_int(rng, 1, kv_max)]) if causal else 0
        return dict(op=op, causal=causal, B=B, new_min=rng.choice([0 if B > 4 else 1, 1, max(1, new_max // 2)]),
                    new_max=new_max, chunks=rng.choice([0, 0, rng.randint(1, B)]),
                    kv_min=rng.choice([0, 1, max(1, kv_max // 2)]), kv_max=kv_max, Hq=Hq, Hkv=Hkv, D=D, window=window,
                    bs=bs, pad=pad)
    if op == "fork":
        n = _log_int(rng, 1, 128)
        kv_max = _log_int(rng, 1, max(1, min(8191, 128 * 2047 * 8 * 128 // (n * Hkv * D))))
        return dict(op=op, R=2 * n + rng.randint(0, 64), n=n, kv_max=kv_max, Hkv=Hkv, D=D, bs=bs)
    if op == "compact":
        R = _log_int(rng, 1, 1024)
        return dict(op=op, R=R, per=_log_int(rng, 1, 65536 // 2 // R), shared=rng.choice([0.0, 0.25, 0.5]), bs=bs)
    n = _log_int(rng, 1, max(1, 8192 * 16 * 8 * 128 // (bs * Hkv * D)))
    n = min(n, 65536)
    return dict(op=op, n=n, blocks=2 * n + rng.randint(0, 99), Hkv=Hkv, D=D, bs=bs)


# ------------------------------------------------------------------ inputs

def _host_ints(seed, salt, lo, hi, n):
    g = torch.Generator().manual_seed(seed * 1000003 + salt)
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _order(seed, salt, n):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed * 1000003 + salt))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _starts(lens):
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)])


def _int32(x):
    return x.to("cuda", torch.int32)


def _tables(seed, lens, bs, spare):
    """A block table in the order an allocator hands blocks out, the blocks left and the pool's size: entries past a
    request's blocks are -1."""
    nb = (lens + bs - 1) // bs
    maxb = max(1, int(nb.max()))
    used = int(nb.sum())
    phys = _order(seed, 5, used + spare)
    table = torch.full((len(lens), maxb), -1, dtype=torch.int64)
    table[torch.arange(maxb)[None, :] < nb[:, None]] = phys[:used]
    return table, phys[used:], used + spare


def _attn_lens(case, seed):
    """New tokens and positions attended of each request. A case has one set of them, so that its outputs' shapes are
    its own; the seed gives their order."""
    B = case["B"]
    new = _host_ints(1, 2, case["new_min"], case["new_max"], B)
    if case["chunks"]:  # so many requests take many tokens, the others one
        new = torch.where(torch.arange(B) < case["chunks"], torch.full_like(new, case["new_max"]),
                          torch.ones_like(new))
    kv = _host_ints(1, 3, case["kv_min"], case["kv_max"], B)
    if case["causal"]:
        kv = kv + new
    order = _order(seed, 4, B)
    return new[order], kv[order]


def _fork_lens(case, seed):
    return _host_ints(1, 3, 1, case["kv_max"], case["n"])[_order(seed, 4, case["n"])]


def prepare(case, seed):
    op = case["op"]
    gen = _gen(seed)
    st = dict(case)
    dev = "cuda"
    if op == "rope":
        N, Hq, Hkv, D, rd, bs = (case[k] for k in ("N", "Hq", "Hkv", "D", "rd", "bs"))
        qkv = _normal((N, Hq + 2 * Hkv, D), gen)
        used = N - case["pad"]
        pos = _host_ints(seed, 1, 0, case["max_pos"] - 1, N)
        pos[used:] = -1
        freq = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
        ang = torch.arange(case["max_pos"], dtype=torch.float64, device=dev)[:, None] * freq
        nblk = (N + bs - 1) // bs + 4
        first = _order(seed, 7, nblk)[:(N + bs - 1) // bs] * bs
        slots = (first[:, None] + torch.arange(bs)[None, :]).reshape(-1)[:N].clone()
        slots[used:] = -1
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], used=used, pos=_int32(pos),
                  cos=ang.cos().float(), sin=ang.sin().float(), slots=slots.to(dev), eps=1e-6,
                  qw=1 + 0.1 * torch.randn(D, generator=gen, device=dev) if case["norm"] else None,
                  kw=1 + 0.1 * torch.randn(D, generator=gen, device=dev) if case["norm"] else None,
                  q_out=torch.zeros((N, Hq, D), dtype=torch.bfloat16, device=dev))
        if case["pool"]:
            pool = torch.zeros((2, nblk, Hkv, bs, D), dtype=torch.bfloat16, device=dev)
            st.update(k_pool=pool[0], v_pool=pool[1])
        else:
            st.update(k_out=torch.zeros((N, Hkv, D), dtype=torch.bfloat16, device=dev))
        return st
    if op == "attn":
        new, kv = _attn_lens(case, seed)
        Hq, Hkv, D, bs = (case[k] for k in ("Hq", "Hkv", "D", "bs"))
        table, _, nblk = _tables(seed, kv, bs, 2)
        N = max(1, int(new.sum()) + case["pad"])
        st.update(q=_normal((N, Hq, D), gen), k_pool=_normal((nblk, Hkv, bs, D), gen),
                  v_pool=_normal((nblk, Hkv, bs, D), gen), table=_int32(table), kv=_int32(kv), cu=_int32(_starts(new)),
                  longest=max(1, int(new.max())), scale=1.0 / math.sqrt(D),
                  out=torch.zeros((N, Hq, D), dtype=torch.bfloat16, device=dev))
        return st
    if op == "fork":
        R, n, Hkv, D, bs = (case[k] for k in ("R", "n", "Hkv", "D", "bs"))
        lens = torch.zeros(R, dtype=torch.int64)
        who = _order(seed, 8, R)
        parents, children = who[:n], who[n:2 * n]
        lens[parents] = _fork_lens(case, seed)
        # the blocks left lie in order on the stack, as they do in a new pool and after a request was dropped
        table, left, nblk = _tables(seed, lens, bs, n + 16)
        left = left.sort().values
        free = torch.full((nblk,), -1, dtype=torch.int64)
        free[:len(left)] = left
        st.update(table=_int32(table), lens=_int32(lens), refs=torch.zeros(nblk, dtype=torch.int32, device=dev),
                  free=_int32(free), count=_int32(torch.tensor([len(left)])),
                  mid=torch.zeros(1, dtype=torch.int32, device=dev),
                  copies=torch.zeros((n, 2), dtype=torch.int32, device=dev), parents=_int32(parents),
                  children=_int32(children), k_pool=_normal((nblk, Hkv, bs, D), gen),
                  v_pool=_normal((nblk, Hkv, bs, D), gen))
        return st
    if op == "compact":
        R, per, bs = case["R"], case["per"], case["bs"]
        nblk = 2 * R * per
        ids = _order(seed, 9, nblk)
        table = ids[:R * per].view(R, per).clone()
        refs = torch.zeros(nblk, dtype=torch.int64)
        # leading blocks that every other request shares with the one before it
        share = int(per * case["shared"])
        if share:
            refs[table[0:R // 2 * 2:2, :share].reshape(-1)] = 1
            dropped = table[1:R // 2 * 2:2, :share].reshape(-1)
            table[1:R // 2 * 2:2, :share] = table[0:R // 2 * 2:2, :share]
            ids = torch.cat([ids, dropped])
        left = ids[R * per:]
        left = left[_order(seed, 10, len(left))]
        free = torch.full((nblk,), -1, dtype=torch.int64)
        free[:len(left)] = left
        lens = per * bs - _host_ints(seed, 11, 0, bs - 1, R)
        st.update(table=_int32(table), lens=_int32(lens), refs=_int32(refs), free=_int32(free),
                  count=_int32(torch.tensor([len(left)])))
        st.update(out=dict(table=torch.zeros_like(st["table"]), refs=torch.zeros_like(st["refs"]),
                           free=torch.zeros_like(st["free"]), count=torch.zeros_like(st["count"]),
                           remap=torch.zeros_like(st["refs"]),
                           moves=torch.zeros((nblk // 2, 2), dtype=torch.int32, device=dev)))
        return st
    n, Hkv, D, bs = (case[k] for k in ("n", "Hkv", "D", "bs"))
    ids = _order(seed, 12, case["blocks"])
    copies = torch.stack([ids[:n], ids[n:2 * n]], dim=1)
    copies[_host_ints(seed, 13, 0, n - 1, n // 16)] = -1  # forks that had nothing to copy
    st.update(copies=_int32(copies), k_pool=_normal((case["blocks"], Hkv, bs, D), gen),
              v_pool=_normal((case["blocks"], Hkv, bs, D), gen))
    return st


# ------------------------------------------------------------- plain forms

def _rotated(x, w, s):
    """x [N, H, D] in 32 bits, normalised by head where w is given, the first rd dims rotated; zeros where the
    position is negative."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + s["eps"]) * w
    rd = s["rd"]
    at = s["pos"].long().clamp(min=0)
    c, sn = s["cos"][at][:, None, :], s["sin"][at][:, None, :]
    if s["pairs"] == "half":
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat([a * c - b * sn, a * sn + b * c], dim=-1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], dim=-1).flatten(-2)
    y = torch.cat([y, x[..., rd:]], dim=-1)
    return torch.where((s["pos"] >= 0)[:, None, None], y, 0.0).to(torch.bfloat16)


def _plain_rope(s):
    q, k = _rotated(s["q"], s["qw"], s), _rotated(s["k"], s["kw"], s)
    if not s["pool"]:
        return q, k
    n, bs = s["used"], s["bs"]
    at = s["slots"][:n]
    s["k_pool"][at // bs, :, at % bs] = k[:n]
    s["v_pool"][at // bs, :, at % bs] = s["v"][:n]
    return q, s["k_pool"], s["v_pool"]


def _plain_attn(s):
    Hq, Hkv, D, T = s["Hq"], s["Hkv"], s["D"], s["longest"]
    G = Hq // Hkv
    cu, kv = s["cu"].long(), s["kv"].long()
    new = cu[1:] - cu[:-1]
    B, N = new.shape[0], s["q"].shape[0]
    i = torch.arange(T, device=cu.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=N - 1)
    q = s["q"].float()[rows].view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    at = s["table"].long().clamp(min=0)
    L = at.shape[1] * s["bs"]
    j = torch.arange(L, device=cu.device)
    k = s["k_pool"][at].float().permute(0, 2, 4, 1, 3).reshape(B, Hkv, D, L)
    v = s["v_pool"][at].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)
    v = torch.where((j[None, :] < kv[:, None])[:, None, :, None], v, 0.0)
    p = torch.matmul(q, k).view(B, Hkv, G, T, L)
    p *= s["scale"]
    end = (kv - new)[:, None] + i[None, :] + 1 if s["causal"] else kv[:, None].expand(B, T)
    hidden = (j[None, None, :] >= end[:, :, None]) | (j[None, None, :] >= kv[:, None, None])
    if s["window"]:
        hidden = hidden | (j[None, None, :] < end[:, :, None] - s["window"])
    p.masked_fill_(hidden[:, None, None], -math.inf)
    top = p.amax(dim=-1, keepdim=True)
    p -= torch.where(top == -math.inf, 0.0, top)
    p.exp_()
    total = p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(B, Hkv, G * T, L), v).view(B, Hkv, G, T, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, D).to(torch.bfloat16)
    t = torch.arange(N, device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    mine = o[(b * T + t - cu[b]).clamp(0, B * T - 1)]
    return torch.where((t < cu[-1])[:, None, None], mine, s["out"])


def _plain_copy(s):
    c = s["copies"].long()
    c = c[c[:, 0] >= 0]
    s["k_pool"][c[:, 1]] = s["k_pool"][c[:, 0]]
    s["v_pool"][c[:, 1]] = s["v_pool"][c[:, 0]]
    return s["k_pool"], s["v_pool"]


def _plain_fork(s):
    bs = s["bs"]
    par, chi, table, refs = s["parents"].long(), s["children"].long(), s["table"], s["refs"]
    n = s["lens"].long()[par]
    e = torch.arange(table.shape[1], device=par.device)[None, :]
    whole = n // bs
    # whole blocks are shared, a last partial one gets a block of its own
    theirs = table[par]
    shared = e < whole[:, None]
    refs.scatter_add_(0, theirs.long().clamp(min=0).flatten(), shared.to(torch.int32).flatten())
    part = n % bs > 0
    before = part.long().cumsum(0) - part.long()
    fresh = s["free"][(s["count"].long() - 1 - before).clamp(min=0)]
    last = e == whole[:, None]
    row = torch.where(shared, theirs, torch.where(last & part[:, None], fresh[:, None], table[chi]))
    src = theirs.gather(1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    s["copies"].copy_(torch.where(part[:, None], torch.stack([src, fresh], dim=1), -1))
    table[chi] = row
    s["lens"][chi] = n.to(torch.int32)
    left = s["count"] - part.sum().to(torch.int32)
    s["mid"].copy_(left)
    _plain_copy(s)
    # the forks are dropped again
    m = s["lens"].long()[chi]
    mine = e < ((m + bs - 1) // bs)[:, None]
    refs.scatter_add_(0, table[chi].long().clamp(min=0).flatten(), -mine.to(torch.int32).flatten())
    gone = torch.nonzero(refs < 0)[:, 0]
    s["free"][left.long() + torch.arange(gone.shape[0], device=par.device)] = gone.to(torch.int32)
    s["count"].copy_(left + gone.shape[0])
    refs.clamp_(min=0)
    table[chi] = torch.where(mine, -1, table[chi])
    s["lens"][chi] = 0
    return s["copies"], s["mid"], table, s["lens"], refs, s["free"], s["count"], s["k_pool"], s["v_pool"]


def _plain_compact(s):
    bs, n = s["bs"], s["refs"].shape[0]
    ids = torch.arange(n, device=s["refs"].device)
    free = torch.zeros(n, dtype=torch.bool, device=ids.device)
    free[s["free"][:int(s["count"])].long()] = True
    used = n - int(free.sum())
    holes, movers = torch.nonzero(free & (ids < used))[:, 0], torch.nonzero(~free & (ids >= used))[:, 0]
    remap = torch.where(free, -1, ids)
    remap[movers] = holes
    moves = torch.full((n // 2, 2), -1, dtype=torch.int32, device=ids.device)
    moves[:holes.shape[0]] = torch.stack([movers, holes], dim=1).to(torch.int32)
    mine = torch.arange(s["table"].shape[1], device=ids.device)[None, :] < ((s["lens"].long() + bs - 1) // bs)[:, None]
    table = torch.where(mine, remap[s["table"].long().clamp(min=0)].to(torch.int32), s["table"])
    refs = torch.where(ids < used, s["refs"], 0)
    refs[holes] = s["refs"][movers]
    stack = torch.where(ids < n - used, n - 1 - ids, s["free"]).to(torch.int32)
    return table, refs, stack, torch.full_like(s["count"], n - used), remap.to(torch.int32), moves


_PLAIN = dict(rope=_plain_rope, attn=_plain_attn, fork=_plain_fork, compact=_plain_compact, copy=_plain_copy)


# ------------------------------------------------------- the library's calls

def _own_rope(g, s):
    more = dict(q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], interleaved=s["pairs"] == "next", q_out=s["q_out"])
    if not s["pool"]:
        return g.qk_norm_rope(s["q"], s["k"], s["pos"], s["cos"], s["sin"], k_out=s["k_out"], **more)
    q = g.kv_append_rope(s["q"], s["k"], s["v"], s["pos"], s["cos"], s["sin"], s["slots"], s["k_pool"], s["v_pool"],
                         **more)
    return q, s["k_pool"], s["v_pool"]


def _own_attn(g, s):
    if s["causal"]:
        return g.gqa_extend_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["kv"], s["cu"], s["scale"],
                                 out=s["out"], window=s["window"] or None)
    return g.gqa_cross_attn(s["q"], s["k_pool"], s["v_pool"], s["table"], s["kv"], s["cu"], s["scale"], out=s["out"])


def _own_fork(g, s):
    g.kv_fork_blocks(s["table"], s["lens"], s["refs"], s["free"], s["count"], s["parents"], s["children"], s["bs"],
                     copies=s["copies"], free_count_out=s["mid"])
    g.kv_copy_blocks(s["k_pool"], s["v_pool"], s["copies"])
    g.kv_free_blocks(s["table"], s["lens"], s["refs"], s["free"], s["mid"], s["children"], s["bs"],
                     free_count_out=s["count"])
    return s["copies"], s["mid"], s["table"], s["lens"], s["refs"], s["free"], s["count"], s["k_pool"], s["v_pool"]


def _own_compact(g, s):
    o = s["out"]
    g.kv_compact_blocks(s["table"], s["lens"], s["refs"], s["free"], s["count"], s["bs"], moves=o["moves"],
                        remap=o["remap"], block_table_out=o["table"], refs_out=o["refs"], free_blocks_out=o["free"],
                        free_count_out=o["count"])
    return o["table"], o["refs"], o["free"], o["count"], o["remap"], o["moves"]


def _own_copy(g, s):
    g.kv_copy_blocks(s["k_pool"], s["v_pool"], s["copies"])
    return s["k_pool"], s["v_pool"]


_OWN = dict(rope=_own_rope, attn=_own_attn, fork=_own_fork, compact=_own_compact, copy=_own_copy)


def run(state):
    if own:
        import grouped_query_kv_gb300 as g
        return _OWN[state["op"]](g, state)
    return _PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and operations that one pass cannot do without: each input read once, each output written once."""
    op = case["op"]
    if op == "rope":
        N, Hq, Hkv, D = case["N"], case["Hq"], case["Hkv"], case["D"]
        used = N - case["pad"]
        heads = Hq + (2 if case["pool"] else 1) * Hkv
        table = min(used, case["max_pos"]) * case["rd"] * 4
        return dict(bytes=2 * used * heads * D * 2 + used * (12 if case["pool"] else 4) + table, flops=0)
    if op == "attn":
        new, kv = _attn_lens(case, 1)
        Hq, Hkv, D, bs, w = (case[k] for k in ("Hq", "Hkv", "D", "bs", "window"))
        pairs = rows = blocks = 0
        for n, m in zip(new.tolist(), kv.tolist()):
            if not n:
                continue
            if case["causal"]:
                ends = range(m - n + 1, m + 1)
                pairs += sum(min(e, w) for e in ends) if w else sum(ends)
                seen = min(m, n + w - 1) if w else m
            else:
                pairs += n * m
                seen = m
            rows += seen
            blocks += (seen + bs - 1) // bs
        tokens = max(1, int(new.sum()))
        return dict(bytes=2 * rows * Hkv * D * 2 + blocks * 4 + case["B"] * 8 + 2 * tokens * Hq * D * 2,
                    flops=4 * pairs * Hq * D)
    if op == "fork":
        n = _fork_lens(case, 1)
        bs, block = case["bs"], case["bs"] * case["Hkv"] * case["D"] * 2
        parts = int((n % bs > 0).sum())
        entries = int(((n + bs - 1) // bs).sum())
        # entries read, shared and written, then read and cleared; a count read and written both times
        return dict(bytes=parts * block * 4 + entries * (4 * 4 + 4 * 4) + case["n"] * 32, flops=0)
    if op == "compact":
        nblk, entries = 2 * case["R"] * case["per"], case["R"] * case["per"]
        # (free list, references and the map, in and out; tables in and out; the moves)
        return dict(bytes=nblk * (2 + 8 + 4 + 4) + entries * 8 + case["R"] * 4 + nblk // 2 * 8, flops=0)
    row = case["Hkv"] * case["bs"] * case["D"] * 2
    kept = case["n"] - case["n"] // 16
    return dict(bytes=kept * row * 4 + case["n"] * 8, flops=0)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs of `run` from the definitions in 64 bits, request by request."""
    def _exact_rope(s):
        rd, used = s["rd"], s["used"]

        def turned(x, w):
            y = x.double().clone()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(dim=-1, keepdim=True) / s["D"] + s["eps"]) * w.double()
            z = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"][:used].long()][:, None, :]
            half = s["pairs"] == "half"
            first, second = (slice(0, rd // 2), slice(rd // 2, rd)) if half else (slice(0, rd, 2), slice(1, rd, 2))
            t = torch.complex(y[:used, :, first], y[:used, :, second]) * z
            y[:used, :, first], y[:used, :, second] = t.real, t.imag
            y[used:] = 0
            return y

        q, k = turned(s["q"], s["qw"]), turned(s["k"], s["kw"])
        if not s["pool"]:
            return q, k
        out = [q]
        at = s["slots"][:used]
        for pool, rows in ((s["k_pool"], k), (s["v_pool"], s["v"].double())):
            nblk, Hkv, bs, D = pool.shape
            flat = pool.double().permute(0, 2, 1, 3).reshape(nblk * bs, Hkv, D)
            flat.index_copy_(0, at, rows[:used])
            out.append(flat.view(nblk, bs, Hkv, D).permute(0, 2, 1, 3))
        return tuple(out)

    def _exact_attn(s):
        G, bs = s["Hq"] // s["Hkv"], s["bs"]
        out = s["out"].double()
        cu = s["cu"].tolist()
        for b, m in enumerate(s["kv"].tolist()):
            a, e = cu[b], cu[b + 1]
            if a == e:
                continue
            if m == 0:
                out[a:e] = 0
                continue
            ids = s["table"][b, :(m + bs - 1) // bs].long()
            place = torch.arange(m - (e - a), m, device=out.device)[:, None]
            far = place - torch.arange(m, device=out.device)[None, :]
            for h in range(s["Hkv"]):
                k = s["k_pool"][ids, h].double().reshape(-1, s["D"])[:m]
                v = s["v_pool"][ids, h].double().reshape(-1, s["D"])[:m]
                for i in range(h * G, h * G + G):
                    x = (s["q"][a:e, i].double() @ k.T) * s["scale"]
                    if s["causal"]:
                        x[(far < 0) | (far >= s["window"]) if s["window"] else far < 0] = -math.inf
                    out[a:e, i] = torch.softmax(x, dim=1) @ v
        return out

    def _exact_fork(s):
        bs = s["bs"]
        table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
        free, left, copies = s["free"].tolist(), int(s["count"]), []
        for p, c in zip(s["parents"].tolist(), s["children"].tolist()):
            lens[c] = lens[p]
            for e in range(lens[p] // bs):
                table[c][e] = table[p][e]
                refs[table[p][e]] += 1
            if lens[p] % bs:
                left -= 1
                table[c][lens[p] // bs] = free[left]
                copies.append([table[p][lens[p] // bs], free[left]])
            else:
                copies.append([-1, -1])
        mid, gone = left, []
        for c in s["children"].tolist():
            for e in range((lens[c] + bs - 1) // bs):
                refs[table[c][e]] -= 1
                if refs[table[c][e]] < 0:
                    gone.append(table[c][e])
                    refs[table[c][e]] = 0
                table[c][e] = -1
            lens[c] = 0
        free[left:left + len(gone)] = sorted(gone)
        pools = []
        for pool in (s["k_pool"], s["v_pool"]):
            after = pool.clone()
            for src, dst in copies:
                if src >= 0:
                    after[dst] = pool[src]
            pools.append(after.double())
        whole = [torch.tensor(x, dtype=torch.int32)
                 for x in (copies, [mid], table, lens, refs, free, [left + len(gone)])]
        return tuple(whole + pools)

    def _exact_compact(s):
        bs, n, count = s["bs"], s["refs"].shape[0], int(s["count"])
        table, lens, refs, stack = (s[k].tolist() for k in ("table", "lens", "refs", "free"))
        free = set(stack[:count])
        used = n - len(free)
        holes = [b for b in range(used) if b in free]
        movers = [b for b in range(used, n) if b not in free]
        remap = [-1 if b in free else b for b in range(n)]
        after = refs[:used] + [0] * (n - used)
        moves = [[-1, -1] for _ in range(n // 2)]
        for i, (src, dst) in enumerate(zip(movers, holes)):
            remap[src] = dst
            after[dst] = refs[src]
            moves[i] = [src, dst]
        for r, m in enumerate(lens):
            for e in range((m + bs - 1) // bs):
                table[r][e] = remap[table[r][e]]
        stack[:n - used] = range(n - 1, used - 1, -1)
        return tuple(torch.tensor(x, dtype=torch.int32) for x in (table, after, stack, [n - used], remap, moves))

    def _exact_copy(s):
        out = []
        for pool in (s["k_pool"], s["v_pool"]):
            after = pool.clone()
            c = s["copies"][s["copies"][:, 0] >= 0].long()
            after.index_copy_(0, c[:, 1], pool.index_select(0, c[:, 0]))
            out.append(after.double())
        return tuple(out)

    s = prepare(case, seed)
    return dict(rope=_exact_rope, attn=_exact_attn, fork=_exact_fork, compact=_exact_compact,
                copy=_exact_copy)[case["op"]](s)
