"""Calls from host threads of the user's own."""
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
