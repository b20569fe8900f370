"""Failure detection of the 8-bit kernels without a GPU fault: with the MMA
warp's polling shortened to one poll a call gives up before its first tile has
arrived, every other role leaves its waits, the device error word says
KVATTN_ERR_TIMEOUT once, and the next call on the same stream and workspace is
the same to the bit as the one before."""
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
    g.set_wait_limit(0)
    yield
    g.set_wait_limit(0)
    g.set_tuning(0, 0)


def _expect_timeout():
    with pytest.raises(g.KvAttnError) as ei:
        g.check_device_error()
    assert ei.value.status == g.KVATTN_ERR_TIMEOUT
    g.check_device_error()


def _gives_up(call, ctas):
    g.set_tuning(0, ctas)
    try:
        want = call().clone()
        g.check_device_error()
        for _ in range(3):
            g.set_wait_limit(1)
            call()
            _expect_timeout()
            g.set_wait_limit(0)
            assert torch.equal(call(), want)
            g.check_device_error()
    finally:
        g.set_wait_limit(0)
        g.set_tuning(0, 0)


# (every number of columns of a pass; ctas > 0: long runs of tiles and split segments)
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 16, 2), (128, 32, 1), (128, 48, 1), (128, 64, 1), (256, 16, 1),
                                      (256, 32, 1), (256, 48, 1)])
@pytest.mark.parametrize("ctas", [0, 3])
def test_a_wait_that_runs_out_reports_a_timeout_and_the_next_call_is_clean(D, Hq, Hkv, ctas):
    gen = torch.Generator(device="cuda").manual_seed(D + Hq)
    lens, bs, L = [700, 0, 300, 2049], 32, 2080
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = [torch.randn((len(lens), Hkv, L, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    q = torch.randn((len(lens), Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    (kc, ks), (vc, vs) = (g.kv_quantize_fp8(r) for r in rows)
    lt = torch.tensor(lens, **i32)
    _gives_up(lambda: g.gqa_decode_attn_fp8(q, kc, vc, ks, vs, lt, 0.1), ctas)
    new = [torch.randn((len(lens), Hkv, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    _gives_up(lambda: g.gqa_decode_step_fp8(q, *new, kc, vc, ks, vs, lt, 0.1), ctas)

    nb = L // bs
    table = torch.as_tensor(np.random.default_rng(1).permutation(len(lens) * nb).reshape(len(lens), nb), **i32)
    codes = [torch.zeros((len(lens) * nb, Hkv, bs, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((len(lens) * nb, Hkv), device="cuda") for _ in range(2)]
    g.kv_append_paged_fp8(*codes, *scales, *(r.transpose(1, 2).reshape(-1, Hkv, D).contiguous() for r in rows), table,
                          torch.zeros(len(lens), **i32), torch.arange(len(lens) + 1, **i32) * L)
    _gives_up(lambda: g.gqa_decode_attn_paged_fp8(q, *codes, *scales, table, lt, 0.1), ctas)
