"""Refusals of the calls around running requests, on the host: each bad
argument is answered before anything touches a device."""
import ctypes

import pytest

import grouped_query_kv_gb300 as g
from grouped_query_kv_gb300 import build as gbuild

P = 0x10000  # aligned, never dereferenced: the checks fail first
INV, UNS = g.KVATTN_ERR_INVALID_ARG, g.KVATTN_ERR_UNSUPPORTED

ROPE = dict(q=P, k=P, positions=P, cos_table=P, sin_table=P, q_weight=P, k_weight=P, q_out=P, k_out=P, N=10, Hq=4,
            Hkv=2, D=128, rope_dim=128, max_pos=100, q_stride=512, k_stride=256, q_out_stride=512,
            k_out_stride=256, eps=1e-6, interleaved=0)
APPEND = dict(q=P, k=P, v=P, positions=P, cos_table=P, sin_table=P, q_weight=P, k_weight=P, slots=P, q_out=P,
              k_pool=P, v_pool=P, N=10, Hq=4, Hkv=2, D=128, rope_dim=64, max_pos=100, q_stride=512, k_stride=256,
              v_stride=256, q_out_stride=512, eps=1e-6, interleaved=1, num_blocks=4, block_size=16)
EXTEND = dict(q=P, k_pool=P, v_pool=P, block_table=P, seq_lens=P, cu_seqlens=P, out=P, B=2, N=10, Hq=4, Hkv=2, D=128,
              q_stride=512, num_blocks=4, block_size=16, max_blocks=3, scale=0.1, window=10)
CROSS = {("kv_lens" if k == "seq_lens" else k): v for k, v in EXTEND.items() if k != "window"}
FORK = dict(block_table=P, seq_lens=P, refs=P, free_blocks=P, free_count=P, parents=P, children=P, copies=P,
            free_count_out=P, n=3, R=5, max_blocks=8, block_size=16, num_blocks=20, num_free=20)
FREE = dict(block_table=P, seq_lens=P, refs=P, free_blocks=P, free_count=P, requests=P, free_count_out=P, n=3, R=5,
            max_blocks=8, block_size=16, num_blocks=20, num_free=20)
COMPACT = dict(block_table=P, seq_lens=P, refs=P, free_blocks=P, free_count=P, block_table_out=P, refs_out=P,
               free_blocks_out=P, free_count_out=P, moves=P, remap=P, R=5, max_blocks=8, block_size=16,
               num_blocks=20, num_free=20)
COPY = dict(k_pool=P, v_pool=P, copies=P, n=3, num_blocks=20, block_bytes=4096)


def _cases():
    calls = dict(qk_norm_rope=ROPE, kv_append_rope=APPEND, gqa_extend_attn=EXTEND, gqa_cross_attn=CROSS,
                 kv_fork_blocks=FORK, kv_free_blocks=FREE, kv_compact_blocks=COMPACT, kv_copy_blocks=COPY)
    for call, args in calls.items():
        for name, v in args.items():
            if v == P:
                if name not in ("q_weight", "k_weight"):  # (which may be null)
                    yield call, args, {name: None}, INV
                yield call, args, {name: P + 2}, INV
        for bs in (0, 8, 24, 1 << 21):
            yield call, args, dict(block_size=bs), UNS
        for name in ("N", "n", "R", "max_blocks", "num_blocks", "num_free", "max_pos", "Hkv", "B", "window"):
            for bad in (0, -1):
                yield call, args, {name: bad}, INV
        yield call, args, dict(N=(1 << 28) + 1), UNS
        yield call, args, dict(R=65536), UNS
        yield call, args, dict(B=65536), UNS
        for scale in (float("nan"), float("inf")):
            yield call, args, dict(scale=scale), INV
        yield call, args, dict(n=(1 << 28) + 1), UNS
        if "R" in args:
            yield call, args, dict(n=65536), UNS
            yield call, args, dict(num_blocks=(1 << 28) + 1), UNS
            yield call, args, dict(num_free=(1 << 28) + 1), UNS
        yield call, args, dict(max_blocks=(1 << 20) + 1), UNS
        for d in (0, 96, 512):
            yield call, args, dict(D=d), INV if d == 0 else UNS
        for rd in (0, 8, 24, 144):
            yield call, args, dict(rope_dim=rd), UNS
        for eps in (-1e-6, float("nan"), float("inf")):
            yield call, args, dict(eps=eps), INV
        yield call, args, dict(Hq=5), INV
        for s in ("q_stride", "k_stride", "v_stride", "q_out_stride", "k_out_stride"):
            for less in (8, -4):
                yield call, args, {s: args.get(s, 8) - less}, INV
            yield call, args, {s: (1 << 38) + 8}, INV
    for name in ("refs", "refs_out", "remap"):
        for call, args in calls.items():
            yield call, args, {name: P + 8}, INV
    for name in ("copies", "moves"):
        for call, args in calls.items():
            yield call, args, {name: P + 4}, INV
    for b in (0, 2, 4098, -16):
        yield "kv_copy_blocks", COPY, dict(block_bytes=b), INV
    yield "kv_copy_blocks", COPY, dict(block_bytes=(1 << 32) + 16), UNS
    yield "kv_copy_blocks", COPY, dict(n=1 << 28, block_bytes=1 << 32), UNS
    yield "kv_copy_blocks", COPY, dict(k_pool=P + 4), INV
    yield "kv_append_rope", APPEND, dict(slots=P + 4), INV
    yield "kv_append_rope", APPEND, dict(num_blocks=1 << 30), UNS
    for call, args in (("gqa_extend_attn", EXTEND), ("gqa_cross_attn", CROSS)):
        yield call, args, dict(num_blocks=1 << 30), UNS
        yield call, args, dict(out=P + 16), INV


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return g.lib()


CASES = [c for c in _cases() if set(c[2]) <= set(c[1])]


@pytest.mark.parametrize("call,args,change,status", CASES,
                         ids=["%s-%s" % (c[0], "-".join("%s=%s" % kv for kv in c[2].items())) for c in CASES])
def test_bad_arguments_are_refused(lib, call, args, change, status):
    a = dict(args, **change)
    sig = g._SIGS[call][1]
    vals = [ctypes.c_void_p(v) if t is ctypes.c_void_p else v for v, t in zip(a.values(), sig)]
    assert getattr(lib, call)(*vals, None) == status
    assert lib.kvattn_last_error().decode() != ""


def test_the_binding_refuses_host_tensors():
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(8, 32)
    with pytest.raises(ValueError, match="CUDA"):
        g.qk_norm_rope(q, q, i, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_append_rope(q, q, q, i, f, f, i.long(), q[None], q[None])
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_fork_blocks(i[None], i, i, i, i[:1], i, i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_free_blocks(i[None], i, i, i, i[:1], i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_compact_blocks(i[None], i, i, i, i[:1], 16)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_copy_blocks(q[None], q[None], i[None])
    with pytest.raises(ValueError, match="CUDA"):
        g.gqa_extend_attn(q, q[None], q[None], i[None], i, i, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        g.gqa_cross_attn(q, q[None], q[None], i[None], i, i, 1.0)
    with pytest.raises(TypeError):
        g.qk_norm_rope([1], q, i, f, f)
