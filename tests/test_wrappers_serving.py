"""Refusals of the serving wrappers that need no GPU: what they check before the device."""
import pytest
import torch

import video_dit_dynamic_token_b200 as lx


def _weights(N=130, K=64):
    return lx.NvFp4Tensor(torch.zeros((N, K // 2), dtype=torch.uint8), torch.zeros(-(-N // 128) * 8 * K, dtype=torch.uint8),
                          torch.ones(1), N, K)


def test_few_row_weights_of_other_types_and_layouts():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensors"):     # all but the device is right
        lx.lx_nvfp4_gemv(x, _weights())
    for name, t in (("codes", torch.zeros((130, 32), dtype=torch.int32)),
                    ("codes", torch.zeros((130, 64), dtype=torch.uint8)[:, ::2]),
                    ("codes", torch.zeros((32, 130), dtype=torch.uint8).t()),
                    ("codes", torch.zeros((129, 32), dtype=torch.uint8)),
                    ("sf", torch.zeros(1024)), ("sf", torch.zeros(2048, dtype=torch.uint8)[::2]),
                    ("sf", torch.zeros(1023, dtype=torch.uint8)),
                    ("gscale", torch.ones(1, dtype=torch.float64)), ("gscale", torch.ones(2)), ("gscale", torch.ones(0))):
        w = _weights()
        setattr(w, name, t)
        with pytest.raises(ValueError, match="W: not the codes"):
            lx.lx_nvfp4_gemv(x, w)
