"""Calls from host threads of the user's own, two at once among them, and a sound call after one that CUDA refused."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def lx():
    import video_dit_dynamic_token_b200 as m
    return m


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen).to(torch.bfloat16).to(DEV)


def _together(calls, turns=3000):
    """The calls, each by a thread of its own, over and over; the statuses other than 0."""
    start, bad = threading.Barrier(len(calls)), []

    def work(call):
        start.wait()
        for _ in range(turns):
            status = call()
            if status != 0:
                bad.append(status)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_few_row_products_of_two_threads(lx):
    """3 and 8 rows are one kernel with different sizes of shared memory."""
    lib = lx._abi.load()
    gen = torch.Generator().manual_seed(1)
    N, K = 256, 5120
    w = lx.lx_nvfp4_quantize(_rand(gen, N, K))
    xs = [_rand(gen, m, K) for m in (3, 8)]
    want = [lx.lx_nvfp4_gemv(x, w) for x in xs]
    got = [torch.zeros_like(y) for y in want]
    ws = [torch.empty(lx.lx_nvfp4_gemv_ws_size(x.shape[0], N, K), dtype=torch.uint8, device=DEV) for x in xs]
    assert all(t.numel() for t in ws)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()

    def call(i):
        x, y, t, s = xs[i], got[i], ws[i], ctypes.c_void_p(streams[i].cuda_stream)
        return lambda: lib.lx_nvfp4_gemv(x.data_ptr(), x.shape[0], K, w.codes.data_ptr(), w.sf.data_ptr(),
                                         w.gscale.data_ptr(), None, N, K, y.data_ptr(), N, t.data_ptr(), t.numel(), s)

    assert _together([call(0), call(1)]) == []
    assert lx.lx_last_device_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode", ["bf16", "int8fp8"])
def test_sparse_attention_of_two_threads(lx, mode):
    """Plans of different size are one kernel with different sizes of shared memory; so is their selection."""
    lib = lx._abi.load()
    gen = torch.Generator().manual_seed(2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for L, keep in ((256, 0.25), (8192, 1.0)):
        q, k, v = (_rand(gen, 1, 1, L, 64) for _ in range(3))
        out, plan = lx.lx_sparse_attn(q, k, v, keep, mode)
        ws = torch.empty(lx.lx_sparse_attn_ws_size(q, keep, mode), dtype=torch.uint8, device=DEV)
        jobs.append((q, k, v, keep, out, plan, torch.zeros_like(out), plan.idx.clone(), ws))
    torch.cuda.synchronize()

    def call(i):
        q, k, v, keep, _, plan, got, _, ws = jobs[i]
        args = [lx.bhld(t) for t in (q, k, v)], plan.c(), lx.bhld(got), ctypes.c_void_p(streams[i].cuda_stream)
        r = ctypes.byref
        return lambda: lib.lx_sparse_attn(*(r(t) for t in args[0]), keep, lx.MODES[mode], r(args[1]), r(args[2]),
                                          ws.data_ptr(), ws.numel(), args[3])

    assert _together([call(0), call(1)], turns=1000) == []
    assert lx.lx_last_device_status() == 0
    for _, _, _, _, out, plan, got, idx, _ in jobs:
        assert torch.equal(got, out) and torch.equal(plan.idx, idx)


def test_a_refused_launch_leaves_no_error_behind(lx):
    """A stream whose capture was broken refuses launches; the next call on another stream is sound and says so."""
    lib = lx._abi.load()
    gen = torch.Generator().manual_seed(3)
    q, k, v = _rand(gen, 1, 4, 9, 64), _rand(gen, 1, 2, 400, 64), _rand(gen, 1, 2, 400, 64)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (9, 400))
    w = lx.lx_nvfp4_quantize(_rand(gen, 256, 512))
    x, y = _rand(gen, 2, 512), torch.zeros((2, 256), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)
    ws = torch.empty(lx.lx_attn_packed_ws_size(q, k, 1), dtype=torch.uint8, device=DEV)
    means = [torch.zeros((1, 4, 1, 64), device=DEV) for _ in range(2)]
    packed = lambda: lx.lx_attn_packed(q, k, v, cu_q, cu_k, out=out, ws=ws)
    few = lambda: lx.lx_nvfp4_gemv(x, w, out=y)
    few(), packed()
    torch.cuda.synchronize()
    want = out.clone(), y.clone()
    broken, good = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    refused = 0
    with torch.cuda.stream(broken):
        graph.capture_begin(capture_error_mode="relaxed")
        try:
            with pytest.raises(RuntimeError):
                broken.synchronize()      # not allowed in a capture: breaks it
            for call in (packed, few):
                with pytest.raises(lx.LxError):
                    call()
                refused += 1
                with torch.cuda.stream(good):
                    sq, sk = lx.bhld(q), lx.bhld(q)
                    assert lib.lx_pool_means(sq, sk, means[0].data_ptr(), means[1].data_ptr(),
                                             ctypes.c_void_p(good.cuda_stream)) == 0
                    packed(), few()
        finally:
            try:
                graph.capture_end()
            except RuntimeError:
                pass
    assert refused == 2
    torch.cuda.synchronize()
    assert lx.lx_last_device_status() == 0
    assert torch.equal(out, want[0]) and torch.equal(y, want[1])


def test_first_call_of_a_thread(lx):
    """A host thread that has made no CUDA call before: its first one is the library's."""
    gen = torch.Generator().manual_seed(1)
    q, k, v = _rand(gen, 1, 4, 9, 64), _rand(gen, 1, 2, 400, 64), _rand(gen, 1, 2, 400, 64)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (9, 400))
    w = lx.lx_nvfp4_quantize(_rand(gen, 256, 512))
    xq, x = lx.lx_nvfp4_quantize(_rand(gen, 2, 512)), _rand(gen, 2, 512)
    plan = lx.lx_sparse_attn_plan(v, v, 0.5)
    ws = torch.empty(lx.lx_attn_packed_ws_size(q, k, 1), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream()
    calls = [(q, lambda o: lx.lx_attn_packed(q, k, v, cu_q, cu_k, out=o, ws=ws)),
             (torch.empty((2, 256), dtype=torch.bfloat16, device=DEV), lambda o: lx.lx_nvfp4_gemv(x, w, out=o)),
             (torch.empty((2, 256), dtype=torch.bfloat16, device=DEV),
              lambda o: lx.lx_nvfp4_gemm(xq, w, out=o, stream=stream)),
             (v, lambda o: lx.lx_attn_bf16(v, k, v, plan, out=o, stream=stream))]
    for like, call in calls:
        want, got, errors = call(torch.zeros_like(like)).clone(), torch.zeros_like(like), []
        torch.cuda.synchronize()

        def work():
            try:
                call(got)
            except Exception as e:
                errors.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert errors == []
        torch.cuda.synchronize()
        assert lx.lx_last_device_status() == 0
        assert torch.equal(got, want)
