"""Calls from several host threads on one stream: each gives the bits that it gives
alone.  (What comes between a call's two launches, and that nothing does, is looked
at without a GPU in test_threads_cpu.py.)"""
import concurrent.futures
import threading

import pytest
import torch

import grouped_query_kv_gb300 as g

from test_gpu_extend import Case, _normal, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from grouped_query_kv_gb300 import build
    build.build()
    g.set_tuning(0, 0)
    g.set_wait_limit(0)


def _together(jobs):
    gate, bad = threading.Barrier(len(jobs)), []

    def work(job):
        try:
            gate.wait()
            job()
        except BaseException as e:
            bad.append(e)

    ts = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad


def _calls():
    """Calls of different sizes that all split their work, as functions of nothing."""
    cases = [Case([1] * 8, [3000 + 7 * i for i in range(8)], 64, 8, 128, 64, seed=1, pad=0, wide=False),
             Case([200, 1, 90], [2500, 1300, 90], 8, 2, 128, 16, seed=2, pad=0, wide=False),
             Case([700], [5000], 16, 1, 256, 64, seed=3, pad=0, wide=False),
             Case([9] * 30, [1000 + i for i in range(30)], 4, 4, 64, 32, seed=4, pad=0, wide=False, causal=False)]
    q, k, v = _normal((3, 32, 128), 5), _normal((3, 4, 4096, 128), 6), _normal((3, 4, 4096, 128), 7)
    lens = _i32([4096, 777, 2000])
    return [c.run for c in cases] + [lambda: g.gqa_decode_attn(q, k, v, lens, 0.09)]


def test_host_threads_on_one_stream():
    calls = _calls()
    want = [f() for f in calls]
    got = [[] for _ in calls]
    torch.cuda.synchronize()

    def job(i):
        for n in range(60):
            got[i].append(calls[i]())
            if n % 10 == 9:  # (the checks below would else wait for all)
                torch.cuda.current_stream().synchronize()

    _together([lambda i=i: job(i) for i in range(len(calls))])
    g.check_device_error()
    for w, outs in zip(want, got):
        assert len(outs) == 60
        for o in outs:
            assert torch.equal(o, w)


_WORKERS = concurrent.futures.ThreadPoolExecutor(max_workers=4)


class _PerThread:
    """The stream of whichever host thread calls (cudaStreamPerThread)."""
    cuda_stream = 2


def test_the_streams_of_host_threads_side_by_side():
    cases = [Case([1] * 8, [3000 + 7 * i for i in range(8)], 64, 8, 128, 64, seed=1, pad=0, wide=False),
             Case([200, 1, 90], [2500, 1300, 90], 8, 2, 128, 16, seed=2, pad=0, wide=False),
             Case([700], [5000], 16, 1, 256, 64, seed=3, pad=0, wide=False),
             Case([9] * 30, [1000 + i for i in range(30)], 4, 4, 64, 32, seed=4, pad=0, wide=False, causal=False)]
    want = [c.run() for c in cases]
    outs = [[torch.zeros_like(w) for _ in range(40)] for w in want]
    torch.cuda.synchronize()

    def job(i):
        gate.wait()
        for o in outs[i]:
            cases[i].run(out=o, stream=_PerThread)
        g.check_device_error(_PerThread)  # (its work is over before the thread is)

    # (threads that stay, and with them their streams)
    gate = threading.Barrier(len(cases))
    for _ in range(2):
        for done in [_WORKERS.submit(job, i) for i in range(len(cases))]:
            done.result()
        torch.cuda.synchronize()
        for w, got in zip(want, outs):
            for o in got:
                assert torch.equal(o, w)
                o.zero_()
        torch.cuda.synchronize()
