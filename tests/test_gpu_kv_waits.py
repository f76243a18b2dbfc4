"""The cache operators' waits, arrival counts and scratch: calls that end without an error code, the same bits every
time, and a call after one that gave up."""
import ctypes
import gc
import threading
import time

import pytest
import torch

from test_gpu_kv import Step, nv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,dt", [(64, "bf16"), (64, "f16"), (128, "bf16"), (128, "f16"), (256, "bf16"), (256, "f16")])
def test_long_walks_end_alike_and_without_an_error_code(nv, dim, dt):  # noqa: F811
    """Long lists of tiles in every tensor-core kernel, call after call: no wait of any role runs out (lanes that poll for
    themselves have to stay within a phase of one another), and the results repeat bit by bit."""
    s = Step(nv, 40, [700, 300], [2500, 100], 8, 4, dim, 64, dt)
    q, table, lengths, offsets = s.rows(8).cuda(), s.i32(s.table), s.i32(s.lengths), s.i32(s.offsets)
    first = nv.kv_attention(q, s.kv, table, lengths, q_offsets=offsets, max_q=700)
    for _ in range(200):
        again = nv.kv_attention(q, s.kv, table, lengths, q_offsets=offsets, max_q=700)
    assert torch.equal(first, again) and torch.isfinite(first).all()
    assert nv.take_device_error() == 0


def spread(nv, seed, new, ctx):  # noqa: F811
    """A step whose heads are split over the whole GPU, and its arguments on the device."""
    s = Step(nv, seed, [new], [ctx], 16 if new == 1 else 4, 2, 128, 64, "bf16")
    q = s.rows(s.heads).cuda()
    return s, q, (s.i32(s.table), s.i32(s.lengths)), dict(q_offsets=s.i32(s.offsets), max_q=new)


@pytest.mark.parametrize("sizes", [[(1, 30000), (1, 21000)], [(300, 3000), (250, 4000)], [(1, 30000), (300, 3000)]])
def test_graphs_of_one_capture_stream_run_at_the_same_time(nv, sizes):  # noqa: F811
    """Two graphs captured on the default capture stream, launched on two streams at once, beside eager calls on a third."""
    steps = [spread(nv, 41 + i, *size) for i, size in enumerate(sizes)]
    want = [nv.kv_attention(q, s.kv, *args, **kw) for s, q, args, kw in steps]
    graphs, outs = [], []
    for s, q, args, kw in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([nv.kv_attention(q, s.kv, *args, **kw) for _ in range(8)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    s, q, args, kw = steps[0]
    for _ in range(10):
        for out in outs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [nv.kv_attention(q, s.kv, *args, **kw) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for out, w in zip(outs, want) for o in out)
        assert all(torch.equal(o, want[0]) for o in eager)
    assert nv.take_device_error() == 0


def test_captures_reuse_the_scratch_of_graphs_that_are_gone(nv):  # noqa: F811
    s, q, args, kw = spread(nv, 43, 1, 30000)
    want = nv.kv_attention(q, s.kv, *args, **kw)
    out = torch.empty_like(want)

    def capture():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.kv_attention(q, s.kv, *args, out=out, **kw)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

    free = []
    for _ in range(12):
        capture()
        gc.collect()
        torch.cuda.synchronize()
        time.sleep(0.05)  # a graph's memory is given back by a thread of the driver's
        free.append(torch.cuda.mem_get_info()[0])
    assert free[3] - free[-1] < 4 << 20  # one workspace is larger


def test_per_thread_default_stream(nv):  # noqa: F811
    """Threads that call on their own per-thread default streams, one handle for all, at the same time."""
    from nvfp4_quantized_matmul_gb300 import binding

    lib = nv.library()
    steps = [spread(nv, 44 + i, 1, 20000 + 3000 * i) for i in range(3)]
    want = [nv.kv_attention(q, s.kv, *args, **kw) for s, q, args, kw in steps]
    outs = [[torch.zeros_like(w) for _ in range(40)] for w in want]
    torch.cuda.synchronize()
    start, status = threading.Barrier(len(steps)), []

    def calls(i):
        s, q, (table, lengths), kw = steps[i]
        batch = binding.KvBatchStruct(table.data_ptr(), table.shape[1], table.stride(0), lengths.data_ptr(), None, 1, 1)
        start.wait()
        for o in outs[i]:
            status.append(lib.nvfp4_kv_attention(s.kv._ref, ctypes.addressof(batch), 2, q.data_ptr(), q.stride(0), s.heads, 1,
                                                 128**-0.5, 0, o.data_ptr(), o.stride(0), 2))  # cudaStreamPerThread

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not any(status)
    assert all(torch.equal(o, w) for out, w in zip(outs, want) for o in out)


STREAM_CODES, CHUNK_CODES = {41, 42, 43}, set(range(51, 67))


@pytest.mark.parametrize("dim,dt", [(64, "f16"), (128, "bf16"), (128, "f16"), (256, "bf16"), (256, "f16")])
@pytest.mark.parametrize("new,ctx", [(1, 30000), (300, 3000)])
def test_a_wait_that_runs_out(nv, opt, new, ctx, dim, dt):  # noqa: F811
    """Every second CTA waits for one arrival too many, so that waits run out after the shortened limit: the call comes back, an error code
    says so, and after that was read the next call is right."""
    s = Step(nv, 47, [new], [ctx], 4, 2, dim, 64, dt)
    q, args, kw = s.rows(4).cuda(), (s.i32(s.table), s.i32(s.lengths)), dict(q_offsets=s.i32(s.offsets), max_q=new)
    want = nv.kv_attention(q, s.kv, *args, **kw)
    torch.cuda.synchronize()
    assert nv.take_device_error() == 0
    opt("wait_limit_us", 1000)
    opt("test_withhold", 1)
    start = time.perf_counter()
    nv.kv_attention(q, s.kv, *args, **kw)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - start
    opt("test_withhold", 0)
    opt("wait_limit_us", 0)
    code = nv.take_device_error()
    assert code in (STREAM_CODES if new == 1 else CHUNK_CODES), code
    assert 0.001 <= elapsed < 1.0
    assert torch.equal(nv.kv_attention(q, s.kv, *args, **kw), want)
    assert nv.take_device_error() == 0


@pytest.mark.parametrize("dim,dt", [(64, "f16"), (128, "bf16"), (256, "bf16"), (256, "f16")])
@pytest.mark.parametrize("new,ctx", [([1], [30000]), ([1] * 40, [211 * j % 4001 for j in range(40)]), ([300], [3000]),
                                     ([200, 150, 40, 1], [100, 1900, 2000, 9000])], ids=lambda v: str(v)[:16])
def test_calls_after_one_that_gave_up(nv, opt, new, ctx, dim, dt):  # noqa: F811
    """What a call that gave up could not finish is no number and the rest is right, and the calls after it on the stream are
    right although nobody has asked for the error: nothing of it is left behind."""
    s = Step(nv, 48, new, ctx, 4, 2, dim, 64, dt)
    q, args, kw = s.rows(4).cuda(), (s.i32(s.table), s.i32(s.lengths)), dict(q_offsets=s.i32(s.offsets), max_q=max(new))
    want = nv.kv_attention(q, s.kv, *args, **kw)
    out = torch.zeros_like(want)
    for _ in range(2):
        opt("wait_limit_us", 1000)
        opt("test_withhold", 1)
        nv.kv_attention(q, s.kv, *args, out=out, **kw)
        opt("test_withhold", 0)
        opt("wait_limit_us", 0)
        lost = torch.isnan(out).all(-1)
        assert lost.any() and torch.equal(out[~lost], want[~lost])
        for _ in range(3):
            assert torch.equal(nv.kv_attention(q, s.kv, *args, **kw), want)
    assert nv.take_device_error() in STREAM_CODES | CHUNK_CODES
    assert nv.take_device_error() == 0
