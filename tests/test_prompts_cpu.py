"""Refusals of the calls that take prompts into a paged cache, on the host:
each bad argument is answered before anything touches a device."""
import ctypes

import pytest

import grouped_query_kv_gb300 as g
from grouped_query_kv_gb300 import build as gbuild

P = 0x10000  # aligned, never dereferenced: the checks fail first
INV, UNS = g.KVATTN_ERR_INVALID_ARG, g.KVATTN_ERR_UNSUPPORTED

TABLES = dict(cached_lens=P, new_lens=P, block_table=P, free_blocks=P, free_count=P, free_count_out=P,
              cu_seqlens=P, slots=P, B=4, max_blocks=8, block_size=16, num_free=10, num_slots=20)
SLOTS = dict(k_pool=P, v_pool=P, k_new=P, v_new=P, slots=P, N=5, Hkv=2, D=64, k_stride=128, v_stride=128,
             num_blocks=4, block_size=16)
PREFILL = dict(q=P, k=P, v=P, cu_seqlens=P, out=P, B=2, N=10, Hq=4, Hkv=2, D=128, q_stride=512,
               k_stride=256, v_stride=256, scale=0.1, window=10)
APPEND8 = dict(k_codes=P, v_codes=P, k_scale=P, v_scale=P, k_new=P, v_new=P, block_table=P, cached_lens=P,
               cu_seqlens=P, B=2, N=10, Hkv=2, D=128, k_stride=256, v_stride=256, num_blocks=4,
               block_size=16, max_blocks=3)
ATTN8 = dict(q=P, k_codes=P, v_codes=P, k_scale=P, v_scale=P, block_table=P, seq_lens=P, out=P, B=2, Hq=4,
             Hkv=2, D=128, num_blocks=4, block_size=16, max_blocks=3, scale=0.1)


def _cases():
    calls = dict(kv_block_tables=TABLES, kv_append_slots=SLOTS, gqa_prefill_attn=PREFILL,
                 kv_append_paged_fp8=APPEND8, gqa_decode_attn_paged_fp8=ATTN8)
    for call, args in calls.items():
        for name, v in args.items():
            if v == P:
                yield call, args, {name: None}, INV
                yield call, args, {name: P + 2}, INV
    for call, args in calls.items():
        if "num_blocks" in args or call == "kv_block_tables":
            for bs in (0, 8, 24, 1 << 21):
                yield call, args, dict(block_size=bs), UNS
        if "scale" in args:
            for s in (float("nan"), float("inf")):
                yield call, args, dict(scale=s), INV
        if "D" in args:
            for d in (0, 96, 512):
                yield call, args, dict(D=d), INV if d == 0 else UNS
            yield call, args, dict(Hkv=0), INV
            yield call, args, dict(Hkv=5000, Hq=5000, k_stride=1 << 20, v_stride=1 << 20, q_stride=1 << 20), UNS
        if "N" in args:
            yield call, args, dict(N=0), INV
            yield call, args, dict(N=-3), INV
            yield call, args, dict(N=(1 << 28) + 1), UNS
        if "B" in args:
            yield call, args, dict(B=0), INV
            yield call, args, dict(B=70000), UNS
        if "max_blocks" in args:
            yield call, args, dict(max_blocks=0), INV
            yield call, args, dict(max_blocks=(1 << 20) + 1), UNS
        if "num_blocks" in args:
            yield call, args, dict(num_blocks=0), INV
        for s in ("q_stride", "k_stride", "v_stride"):
            if s in args:
                for bad in (0, args[s] - 8, args[s] + 4, (1 << 38) + 8):
                    yield call, args, {s: bad}, INV
    yield "kv_block_tables", TABLES, dict(num_free=0), INV
    yield "kv_block_tables", TABLES, dict(num_slots=0), INV
    yield "kv_block_tables", TABLES, dict(num_slots=(1 << 28) + 1), UNS
    yield "kv_block_tables", TABLES, dict(slots=P + 4), INV
    yield "kv_append_slots", SLOTS, dict(slots=P + 4), INV
    yield "kv_append_slots", SLOTS, dict(num_blocks=1 << 30, Hkv=4, k_stride=256, v_stride=256), UNS
    yield "gqa_prefill_attn", PREFILL, dict(out=P + 16), INV
    yield "gqa_prefill_attn", PREFILL, dict(window=0), INV
    yield "gqa_prefill_attn", PREFILL, dict(Hq=5, q_stride=640), INV
    yield "kv_append_paged_fp8", APPEND8, dict(block_size=2048), UNS
    yield "gqa_decode_attn_paged_fp8", ATTN8, dict(block_size=2048), UNS
    yield "gqa_decode_attn_paged_fp8", ATTN8, dict(D=64), UNS


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return g.lib()


CASES = [c for c in _cases() if set(c[2]) <= set(c[1]) or "Hq" in c[2]]


@pytest.mark.parametrize("call,args,change,status", CASES,
                         ids=["%s-%s" % (c[0], "-".join("%s=%s" % kv for kv in c[2].items())) for c in CASES])
def test_bad_arguments_are_refused(lib, call, args, change, status):
    a = dict(args)
    a.update({k: v for k, v in change.items() if k in args})
    sig = g._SIGS[call][1]
    vals = [ctypes.c_void_p(v) if t is ctypes.c_void_p else v for v, t in zip(a.values(), sig)]
    assert getattr(lib, call)(*vals, None) == status
    assert lib.kvattn_last_error().decode() != ""


def test_the_binding_refuses_host_tensors_types_and_shapes():
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.gqa_prefill_attn(q, q, q, cu, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_append_slots(q[None], q[None], q, q, cu.long())
    with pytest.raises(ValueError, match="CUDA"):
        g.kv_block_tables(cu, cu, cu[None], cu, cu[:1], 16, 4)
    with pytest.raises(TypeError):
        g.gqa_prefill_attn([1], q, q, cu, 1.0)
