"""Calls on several host threads are independent: threads that call one kernel with different amounts of
shared memory at the same time each get what they get alone."""
import ctypes
import threading

import pytest
import torch

from test_gpu_selective import cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd(cuda_device):
    from structured_state_space_fwd_b200 import build
    build.build()
    import structured_state_space_fwd_b200 as m
    return m


def together(calls, times=4000):
    """Runs each (entry point, arguments) `times` times on a thread of its own, all at once, and returns
    the status codes that were not 0. ctypes lets the others run during a call."""
    failed, start = [], threading.Barrier(len(calls))

    def loop(fn, args):
        start.wait(timeout=60)
        bad = 0
        for _ in range(times):
            st = fn(*args)
            if st:
                bad += 1
                code = st
        if bad:
            failed.append((fn.__name__, code, bad))
    threads = [threading.Thread(target=loop, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


@pytest.mark.parametrize("T,D,dtype,few,many", [
    (66, 16, "bf16", 16, 256),         # few channels: one block of states, and as many as there are
    (520, 16, "f32", 17, 256),         # clusters
    (16, 16, "f32", 209, 256),         # blocks of states, uncut
])
def test_selective_scan(ssd, monkeypatch, T, D, dtype, few, many):
    from structured_state_space_fwd_b200 import _block
    calls, kept, raw = [], [], []
    real = _block._call

    def note(name, t, stream, *args):
        raw.append((name, args))
        real(name, t, stream, *args)
    monkeypatch.setattr(_block, "_call", note)
    for N in (few, many) * 2:
        d = cuda(inputs(1, T, D, 1, N, dtype, seed=N))
        y, fin, stream = torch.zeros_like(d["u"]), torch.zeros_like(d["initial_states"]), torch.cuda.Stream()
        expect = ssd.ssd_selective_scan(**d, return_final_states=True)
        stream.wait_stream(torch.cuda.current_stream())
        ssd.ssd_selective_scan(**d, y=y, final_states=fin, stream=stream)
        name, args = raw[-1]
        calls.append((getattr(ssd.lib(), name), (*args, stream.cuda_stream)))
        kept.append((d, y, fin, stream, expect))
    torch.cuda.synchronize()
    for _, y, fin, _, _ in kept:
        y.zero_(), fin.zero_()
    torch.cuda.synchronize()
    assert together(calls) == []
    for _, y, fin, _, expect in kept:
        assert torch.equal(y, expect[0]) and torch.equal(fin, expect[1])


def test_chunk_steps(ssd):
    """The cumulative sums and the scan of a chunk in fp32, with the smallest and the largest chunks and states."""
    calls, kept = [], []
    for Q, P, N in ((16, 4, 4), (256, 256, 256)) * 2:
        b, T, H = 1, Q, 1
        shape = ssd.ShapeT(b, T, H, P, 1, N, Q, 0, 0)
        g = torch.Generator().manual_seed(Q)

        def new(*s):
            return torch.randn(*s, generator=g).cuda()
        x, dt, A, B, C = new(b, T, H, P), new(b, T, H).abs() * 0.1, -new(H).abs(), new(b, T, 1, N), new(b, T, 1, N)
        cs = ssd.ssd_chunk_cumsum(dt, A, Q, shape)
        entry = new(b, 1, H, P, N)
        y = ssd.ssd_chunk_scan(x, dt, B, C, None, cs, entry, shape)
        cs1, y1, stream = torch.zeros_like(cs), torch.zeros_like(y), torch.cuda.Stream()
        p = [t.data_ptr() for t in (x, dt, B, C)]
        lib, ref = ssd.lib(), ctypes.byref(shape)
        calls.append((lib.ssd_chunk_cumsum, (ref, p[1], A.data_ptr(), cs1.data_ptr(), stream.cuda_stream)))
        calls.append((lib.ssd_chunk_scan, (ref, *p, None, cs.data_ptr(), entry.data_ptr(), y1.data_ptr(),
                                           stream.cuda_stream)))
        kept.append((x, dt, A, B, C, cs, entry, y, cs1, y1, stream, shape))
    torch.cuda.synchronize()
    assert together(calls) == []
    for *_, cs, entry, y, cs1, y1, stream, shape in kept:
        assert torch.equal(cs, cs1) and torch.equal(y, y1)
