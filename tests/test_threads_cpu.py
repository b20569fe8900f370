"""Calls from several host threads, without a GPU: the library's host side over a
stand-in for the CUDA runtime (fake_cudart.cpp) that writes down every launch and
allocation.  A call whose partial results go through a workspace launches two
kernels; between them nothing else may use that workspace."""
import ctypes
import os
import subprocess
import threading

import pytest

import grouped_query_kv_gb300 as g
from grouped_query_kv_gb300 import build as gbuild

HERE = os.path.dirname(os.path.abspath(__file__))
P = 0x100000  # aligned, never dereferenced

# name -> arguments before the stream, for a batch of B (and D = 128 where not said)
CALLS = {
    "gqa_decode_attn": lambda B: (P, P, P, P, P, B, 32, 4, 128, 512, 0.1),
    "gqa_decode_attn_window": lambda B: (P, P, P, P, P, B, 32, 4, 64, 512, 0.1, 100),
    "gqa_decode_attn_multi": lambda B: (P, P, P, P, P, B, 3, 32, 4, 128, 512, 0.1),
    "gqa_decode_step": lambda B: (P, P, P, P, P, P, P, B, 32, 4, 256, 512, 0.1),
    "gqa_decode_attn_paged": lambda B: (P, P, P, P, P, P, B, 1, 32, 4, 128, 64, 16, 8, 0.1),
    "gqa_decode_attn_fp8": lambda B: (P, P, P, P, P, P, P, B, 32, 4, 128, 512, 0.1),
    "gqa_decode_attn_paged_fp8": lambda B: (P, P, P, P, P, P, P, P, B, 32, 4, 128, 64, 16, 8, 0.1),
    "gqa_decode_attn_noalloc": lambda B: (P, P, P, P, P, B, 32, 4, 128, 512, 0.1),
    "gqa_extend_attn": lambda B: (P, P, P, P, P, P, P, B, 3 * B, 32, 4, 128, 4096, 64, 16, 8, 0.1, 1000),
    "gqa_cross_attn": lambda B: (P, P, P, P, P, P, P, B, 40 * B, 4, 4, 64, 256, 64, 16, 8, 0.1),
}


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gbuild.build()
    objs = [os.path.join(gbuild.BUILD, os.path.basename(s)[:-3] + ".o") for s in gbuild.sources()]
    if not all(map(os.path.exists, objs)):
        gbuild.build(force=True)
    so = str(tmp_path_factory.mktemp("fake") / "libkvattn_fake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(gbuild.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", "-Wl,-Bsymbolic", "-Wl,-z,defs",
                    "-I", cuda, os.path.join(HERE, "fake_cudart.cpp"), *objs, "-o", so], check=True)
    h = ctypes.CDLL(so)
    for name, (res, args) in g._SIGS.items():
        getattr(h, name).restype, getattr(h, name).argtypes = res, args
    h.fake_log.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
    h.fake_log.restype = ctypes.c_size_t
    h.fake_capture.argtypes = [ctypes.c_ulonglong]
    h.fake_capture.restype = h.fake_thread.restype = h.fake_clear.restype = None
    yield h
    h.fake_capture(0)


@pytest.fixture(autouse=True)
def _clean(lib):
    lib.fake_capture(0)
    lib.kvattn_release()
    lib.fake_clear()


def _log(lib, word):
    buf = ctypes.create_string_buffer(1 << 20)
    assert lib.fake_log(buf, len(buf)) <= len(buf)
    return [line.split() for line in buf.value.decode().splitlines() if line.startswith(word)]


def _together(lib, jobs):
    """jobs[i]() in host thread i, all at once; their exceptions."""
    gate, bad = threading.Barrier(len(jobs)), []

    def work(i):
        try:
            lib.fake_thread(i)
            gate.wait()
            jobs[i]()
        except BaseException as e:  # (pytest sees it in the main thread)
            bad.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


def _call(lib, name, B, stream):
    assert getattr(lib, name)(*CALLS[name](B), stream) == g.KVATTN_OK, lib.kvattn_last_error()


def _joined_in_pairs(launches):
    """Each split kernel's launch is followed by its own thread's join."""
    assert launches and len(launches) % 2 == 0
    for first, then in zip(launches[::2], launches[1::2]):
        assert "merge_kernel" not in first[3] and "combine_kernel" not in first[3], launches
        assert "merge_kernel" in then[3] or "combine_kernel" in then[3], launches
        assert first[1] == then[1], launches


@pytest.mark.parametrize("captured", [0, 7])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_s_launches_on_one_stream_stay_together(lib, name, captured):
    if captured and name == "gqa_decode_attn_noalloc":
        _call(lib, name, 2, 0x500)  # (its first call may not be captured)
        lib.fake_clear()
    lib.fake_capture(captured)
    _together(lib, [lambda B=B: [_call(lib, name, B, 0x500) for _ in range(3)] for B in (2, 5, 9, 17)])
    _joined_in_pairs(_log(lib, "launch"))


def test_different_calls_on_one_stream_stay_together(lib):
    # (gqa_decode_attn_noalloc has an array of its own, not the stream's workspace)
    names = sorted(set(CALLS) - {"gqa_decode_attn_noalloc"})
    _together(lib, [lambda n=n: [_call(lib, n, 4, 0x500) for _ in range(2)] for n in names])
    _joined_in_pairs(_log(lib, "launch"))


def test_calls_on_two_streams_do_not_wait_for_each_other(lib):
    names = ["gqa_extend_attn", "gqa_decode_attn"]
    _together(lib, [lambda s=s: [_call(lib, n, 4, s) for n in names * 3] for s in (0x500, 0x600)])
    launches = _log(lib, "launch")
    for s in ("1280", "1536"):
        _joined_in_pairs([x for x in launches if x[2] == s])
    order = [x[2] for x in launches]
    assert any(a != b for a, b in zip(order[::2], order[1::2])), order  # (some came between)
    assert len(_log(lib, "malloc")) >= 2


def test_release_waits_for_the_calls_under_way(lib):
    # (a workspace is not freed between a call's two launches)
    done = threading.Event()

    def calls(s):
        try:
            for n in ("gqa_extend_attn", "gqa_decode_attn", "gqa_decode_attn_paged_fp8"):
                _call(lib, n, 4, s)
        finally:
            done.set()

    def release():
        while not done.is_set():
            lib.kvattn_release()

    _together(lib, [lambda: calls(0x500), lambda: calls(0x700), release, release])
    lines, open_calls = _log(lib, ""), {}
    for x in lines:
        if x[0] == "launch" and "merge_kernel" not in x[3] and "combine_kernel" not in x[3]:
            open_calls[x[1]] = x
        elif x[0] == "launch":
            del open_calls[x[1]]
        elif x[0] == "free":
            assert not open_calls, (x, open_calls)
    assert any(x[0] == "free" for x in lines)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_first_call_of_a_host_thread(lib, name):
    # a thread has no context until a runtime call that needs one; the maps' encoding, a
    # driver call, is refused without
    _call(lib, name, 4, 0x500)  # (so that the thread's call has nothing to allocate)
    _together(lib, [lambda: _call(lib, name, 4, 0x500)])


def test_the_first_call_of_a_host_thread_that_needs_no_workspace(lib):
    _together(lib, [lambda: _prefill(lib)])


def _prefill(lib):
    # (through internal maps too)
    rc = lib.gqa_prefill_attn(P, P, P, P, P, 2, 100, 32, 4, 128, 4096, 512, 512, 0.1, 1000, 0x500)
    assert rc == g.KVATTN_OK, lib.kvattn_last_error()


@pytest.mark.parametrize("captured", [0, 7])
@pytest.mark.parametrize("name", sorted(set(CALLS) - {"gqa_decode_attn_noalloc"}))
def test_the_stream_of_each_host_thread_has_a_workspace_of_its_own(lib, name, captured):
    # (one handle, a stream in each host thread: their calls run side by side)
    per_thread = 2
    lib.fake_capture(captured)
    _together(lib, [lambda: [_call(lib, name, 4, per_thread) for _ in range(3)] for _ in range(3)])
    assert sorted(x[1] for x in _log(lib, "malloc")) == ["0", "1", "2"]
    launches = _log(lib, "launch")
    for t in "012":
        _joined_in_pairs([x for x in launches if x[1] == t])
    # and they do not wait for each other
    assert any(a[1] != b[1] for a, b in zip(launches[::2], launches[1::2])), launches


def test_release_frees_nothing_beside_work(lib):
    # (cudaFree waits for the device's work as well, but is kept from meeting any)
    for name in ("gqa_extend_attn", "gqa_decode_attn"):
        for s in (0x500, 0x600):
            _call(lib, name, 4, s)
    lib.fake_clear()
    lib.kvattn_release()
    words = [x[0] for x in _log(lib, "")]
    assert words[0] == "sync" and words.count("free") >= 2 and set(words[1:]) == {"free"}
    lib.fake_clear()
    lib.kvattn_release()
    assert not _log(lib, "")  # (nothing is held, nothing is waited for)
