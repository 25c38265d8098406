"""The serving operators together, as a decoder uses them: prompts in one packed call, then
one token a sequence (few-row projections, cache, attention, few-row projection), eagerly and as
a replayed graph, with caches of their own and behind a shared prompt.

Every stage is held to the fp64 oracle of its own bf16 inputs, with the bounds of
test_gpu_packed.py and test_gpu_gemv.py, so that errors do not add up along the chain."""
import types

import numpy as np
import pytest
import torch

import oracle
from oracle import nvfp4_ref as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, HID = 8, 2, 64, 512


@pytest.fixture(scope="module")
def lx():
    import video_dit_dynamic_token_b200 as m
    return m


def _i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def _rand(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16).to(DEV)


def _heads(t, lo, n):
    """[T, *] columns lo .. lo + n D as [1, n, T, D] (a view)."""
    return t[:, lo:lo + n * D].unflatten(1, (n, D)).transpose(0, 1).unsqueeze(0)


def _np(t):
    return t[0].float().cpu().numpy()


def _check_attn(out, lse, ref):
    bo, bl = oracle.packed_attn_bounds(ref, D)
    live = ~np.isnan(ref["keys"])
    o, l = _np(out), lse.cpu().numpy()
    assert np.all(np.abs(o - ref["o"])[live] <= bo[live])
    seen = live & np.isfinite(ref["lse"])
    assert np.all(np.abs(l - ref["lse"])[seen] <= bl[seen])


def _check_rows(y, x, wr, bias):
    """Bounds of few-row products: eight or fewer rows, all elements within 2^-35 of the largest."""
    x = x.float().cpu().numpy().astype(np.float64)
    a = np.abs(x)
    assert x.shape[0] <= 8 and a[a > 0].min() > 2.0 ** -35 * a.max()
    b = bias.cpu().numpy().astype(np.float64)
    ref = oracle.gemv_nvfp4_ref(x, wr, b)
    bound = 2.0 ** -8 * np.abs(ref["y"]) + (x.shape[1] / 8 + 50) * 2.0 ** -23 * (4 * ref["mag"] + np.abs(b)) + 1e-38
    assert np.all(np.abs(y.float().cpu().numpy() - ref["y"]) <= bound)


@pytest.fixture(scope="module")
def layer(lx):
    """Weights of an attention layer: [Q | K | V] and the output projection, with their oracle forms."""
    gen = torch.Generator().manual_seed(71)
    p = types.SimpleNamespace()
    for name, n in (("qkv", (HQ + 2 * HKV) * D), ("o", HID)):
        w = _rand(gen, n, HID, scale=0.05)
        setattr(p, name, lx.lx_nvfp4_quantize(w))
        setattr(p, name + "_ref", nv.quant_nvfp4_ref(w.float().cpu().numpy()))
        setattr(p, name + "_bias", (torch.randn(n, generator=gen) * 0.1).to(DEV))
    return p


class _Cache:
    """n slots of `cap` keys; used[i] keys of slot i are filled."""

    def __init__(self, n, cap):
        self.K, self.V = (torch.full((1, HKV, n * cap, D), float("nan"), dtype=torch.bfloat16, device=DEV)
                          for _ in range(2))
        self.cu = _i32(i * cap for i in range(n + 1))
        self.used = _i32([0] * n)

    def add(self, k, v):
        """One key a slot, at the place that the lengths on the device say."""
        at = (self.cu[:-1] + self.used).long()
        self.K.index_copy_(2, at, k)
        self.V.index_copy_(2, at, v)
        self.used += 1


def _prompts(lx, layer, lens, cache, gen):
    """The prompts' attention in one packed call; fills the cache."""
    cu = np.concatenate(([0], np.cumsum(lens)))
    qkv = lx.lx_nvfp4_gemm(lx.lx_nvfp4_quantize(_rand(gen, cu[-1], HID)), layer.qkv, bias=layer.qkv_bias)
    q, k, v = _heads(qkv, 0, HQ), _heads(qkv, HQ * D, HKV), _heads(qkv, (HQ + HKV) * D, HKV)
    lse = torch.empty((HQ, int(cu[-1])), device=DEV)
    out = lx.lx_attn_packed(q, k, v, _i32(cu), _i32(cu), lse=lse)
    assert lx.lx_last_device_status() == 0
    _check_attn(out, lse, oracle.packed_attn_ref(_np(q), _np(k), _np(v), cu, cu, True, D ** -0.5))
    if cache is not None:
        starts = cache.cu.tolist()
        for i, n in enumerate(lens):
            cache.K[:, :, starts[i]:starts[i] + n] = k[:, :, cu[i]:cu[i + 1]]
            cache.V[:, :, starts[i]:starts[i] + n] = v[:, :, cu[i]:cu[i + 1]]
        cache.used.copy_(_i32(lens))
    return k, v


def _token(lx, layer, x, cache, prefix=None):
    """One token a sequence: (qkv, attention, lse, layer output)."""
    n = x.shape[0]
    qkv = lx.lx_nvfp4_gemv(x, layer.qkv, bias=layer.qkv_bias)
    cache.add(_heads(qkv, HQ * D, HKV), _heads(qkv, (HQ + HKV) * D, HKV))
    o = torch.empty((n, HQ * D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((HQ, n), device=DEV)
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    q = _heads(qkv, 0, HQ)
    kw = dict(len_k=cache.used, out=_heads(o, 0, HQ), lse=lse)
    if prefix is None:
        lx.lx_attn_packed(q, cache.K, cache.V, cu, cache.cu, **kw)
    else:
        lx.lx_attn_prefix(q, *prefix, cache.K, cache.V, cu, cache.cu, **kw)
    return qkv, o, lse, lx.lx_nvfp4_gemv(o, layer.o, bias=layer.o_bias)


def _check_token(layer, x, cache, got, prefix=None):
    qkv, o, lse, y = got
    n = x.shape[0]
    _check_rows(qkv, x, layer.qkv_ref, layer.qkv_bias)
    ref = oracle.packed_attn_ref(_np(_heads(qkv, 0, HQ)), _np(cache.K), _np(cache.V), range(n + 1), cache.cu.tolist(), True,
                                 D ** -0.5, cache.used.tolist(), *([_np(t) for t in prefix] if prefix else []))
    _check_attn(_heads(o, 0, HQ), lse, ref)
    _check_rows(y, o, layer.o_ref, layer.o_bias)


@pytest.mark.parametrize("lens", [[5, 130, 64], [1], [300, 1, 2, 129, 128, 7]])
def test_prompts_then_tokens(lx, layer, lens):
    gen = torch.Generator().manual_seed(len(lens))
    cache = _Cache(len(lens), 320)
    _prompts(lx, layer, lens, cache, gen)
    x = _rand(gen, len(lens), HID)
    for _ in range(3):
        got = _token(lx, layer, x, cache)
        assert lx.lx_last_device_status() == 0
        _check_token(layer, x, cache, got)
        x = got[3]


@pytest.mark.parametrize("shared", [False, True])
def test_replayed_steps_equal_eager_ones(lx, layer, shared):
    n, steps = 4, 5
    gen = torch.Generator().manual_seed(9)
    prefix = _prompts(lx, layer, [700], None, gen) if shared else None
    lens = [0] * n if shared else [200, 3, 77, 256]

    def start():
        cache = _Cache(n, 300)
        if not shared:
            _prompts(lx, layer, lens, cache, torch.Generator().manual_seed(10))
        return cache, _rand(torch.Generator().manual_seed(11), n, HID)

    cache, x = start()
    eager = []
    for _ in range(steps):
        got = _token(lx, layer, x, cache, prefix)
        _check_token(layer, x, cache, got, prefix)
        eager.append(got)
        x = got[3]
    again, x = start()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = _token(lx, layer, x, again, prefix)
        x.copy_(got[3])
    for k in range(steps):
        g.replay()
        torch.cuda.synchronize()
        assert lx.lx_last_device_status() == 0
        for a, b in zip(got, eager[k]):
            assert torch.equal(a, b)
    assert torch.equal(again.used, cache.used)


def test_shared_prompt_equals_its_copies(lx, layer):
    """Tokens behind a shared prompt, and over caches that each hold a copy of it."""
    n, pre = 3, 137
    gen = torch.Generator().manual_seed(12)
    k, v = _prompts(lx, layer, [pre], None, gen)
    own, copies = _Cache(n, 40), _Cache(n, 180)
    for i, a in enumerate(copies.cu.tolist()[:-1]):
        copies.K[:, :, a:a + pre], copies.V[:, :, a:a + pre] = k, v
    copies.used.fill_(pre)
    x = _rand(gen, n, HID)
    for _ in range(3):
        a, b = _token(lx, layer, x, own, (k, v)), _token(lx, layer, x, copies)
        assert lx.lx_last_device_status() == 0
        assert torch.equal(a[0], b[0])
        _check_token(layer, x, own, a, (k, v))
        _check_token(layer, x, copies, b)
        x = a[3]


def test_streams_given_by_hand(lx, layer):
    """stream=: results and workspaces belong to it, also when much is in flight on both streams."""
    gen = torch.Generator().manual_seed(13)
    n = 3
    x = _rand(gen, n, HID)
    q, k, v = _rand(gen, 1, HQ, n, D), _rand(gen, 1, HKV, n * 600, D), _rand(gen, 1, HKV, n * 600, D)
    cq, ck = _i32(range(n + 1)), _i32(600 * i for i in range(n + 1))
    y0 = lx.lx_nvfp4_gemv(x, layer.qkv, bias=layer.qkv_bias)
    o0 = lx.lx_attn_packed(q, k, v, cq, ck)
    p0 = lx.lx_attn_prefix(q, k, v, k, v, cq, ck)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((lx.lx_nvfp4_gemv(x, layer.qkv, bias=layer.qkv_bias, stream=s),
                    lx.lx_attn_packed(q, k, v, cq, ck, stream=s), lx.lx_attn_prefix(q, k, v, k, v, cq, ck, stream=s)))
        torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)   # would take over a workspace of the wrong stream
    torch.cuda.synchronize()
    assert lx.lx_last_device_status() == 0
    for y, o, p in got:
        assert torch.equal(y, y0) and torch.equal(o, o0) and torch.equal(p, p0)


def test_wrappers_refuse(lx, layer):
    gen = torch.Generator().manual_seed(14)
    q, k, v = _rand(gen, 1, HQ, 4, D), _rand(gen, 1, HKV, 9, D), _rand(gen, 1, HKV, 9, D)
    cq, ck = _i32([0, 1, 4]), _i32([0, 3, 9])
    call = lx.lx_attn_packed
    elsewhere = types.SimpleNamespace(device_index=q.get_device() + 1)
    for args, kw in (((q, k, v, cq.long(), ck), {}), ((q, k, v, cq, ck[:2]), {}), ((q, k, v, cq, ck[None]), {}),
                     ((q, k, v, cq, _i32(range(6))[::2]), {}), ((q, k, v, cq, ck), {"len_k": ck}),
                     ((q.float(), k, v, cq, ck), {}), ((q, k[0], v, cq, ck), {}), ((q, k, v.transpose(2, 3), cq, ck), {}),
                     ((q, k, v, cq, ck), {"lse": torch.empty((HQ, 5), device=DEV)}),
                     ((q, k, v, cq, ck), {"lse": torch.empty((HQ, 4), device=DEV, dtype=torch.float64)}),
                     ((q, k, v, cq.cpu(), ck), {}), ((q, k, v, cq, ck), {"stream": elsewhere})):
        with pytest.raises(ValueError):
            call(*args, **kw)
    for args, kw in (((q, k, v[:, :, :8], cq, ck), {}), ((q, k, v, cq, ck), {"out": q[:, :, :3]}),
                     ((q, k, v, cq, ck), {"scale": 0.0}), ((q, k, v, cq[:1], ck[:1]), {}),
                     ((q[:, :3], k, v, cq, ck), {})):
        with pytest.raises(lx.LxError):
            call(*args, **kw)
    with pytest.raises(lx.LxError):   # a prefix of other heads
        lx.lx_attn_prefix(q, q, q, k, v, cq, ck)
    with pytest.raises(lx.LxError):   # too small a workspace
        lx.lx_attn_prefix(q, k, v, k, v, cq, ck, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    x = _rand(gen, 2, HID)
    for args, kw in (((x.float(), layer.o), {}), ((x.t(), layer.o), {}), ((x[:, :256], layer.o), {}),
                     ((x, layer.o), {"bias": layer.qkv_bias}), ((x, layer.o), {"bias": layer.o_bias.half()}),
                     ((x, layer.o), {"out": x[:1]}), ((x, layer.o), {"out": x.float()}), ((x.cpu(), layer.o), {}),
                     ((x, layer.o), {"stream": elsewhere}),
                     ((x, lx.NvFp4Tensor(layer.o.codes[:1], layer.o.sf, layer.o.gscale, HID, HID)), {})):
        with pytest.raises(ValueError):
            lx.lx_nvfp4_gemv(*args, **kw)
    with pytest.raises(lx.LxError):
        lx.lx_nvfp4_gemv(_rand(gen, 17, HID), layer.o)
    assert lx.lx_last_device_status() == 0


def test_captured_between_streams(lx, layer):
    """A captured call behind a copy, behind work of two streams, and in front of work on another one."""
    gen = torch.Generator().manual_seed(15)
    n = 3
    x, x2 = _rand(gen, n, HID), _rand(gen, n, HID)
    q, k, v = _rand(gen, 1, HQ, n, D), _rand(gen, 1, HKV, n * 600, D), _rand(gen, 1, HKV, n * 600, D)
    cq, ck = _i32(range(n + 1)), _i32(600 * i for i in range(n + 1))
    kc, xc = torch.zeros_like(k), torch.zeros_like(x)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        kc.copy_(k)                                       # a copy in front
        side.wait_stream(main)
        with torch.cuda.stream(side):
            xc.copy_(x)
            a = lx.lx_nvfp4_gemv(xc, layer.qkv, bias=layer.qkv_bias)
        b = lx.lx_attn_packed(q, kc, v, cq, ck)
        main.wait_stream(side)                            # two streams in front
        c = lx.lx_attn_prefix(q, kc, v, kc, v, cq, ck)
        side.wait_stream(main)
        with torch.cuda.stream(side):                     # on another stream behind
            d = lx.lx_nvfp4_gemv(x2, layer.qkv, bias=layer.qkv_bias)
            e = lx.lx_attn_packed(c, kc, v, cq, ck)
        main.wait_stream(side)
        return a, b, c, d, e

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        want = work()
    main.synchronize()
    assert lx.lx_last_device_status() == 0
    plain = lx.lx_attn_packed(want[2], k, v, cq, ck)
    assert torch.equal(plain, want[4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        got = work()
    for _ in range(3):
        for t in (*got, kc, xc):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert lx.lx_last_device_status() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
