"""Products of few bf16 rows with NVFP4 weights (lx_nvfp4_gemv) against the fp64
oracle.

Bound: |Y - y| <= 2^-8 |y| (bf16) + c 2^-23 (4 mag + |bias|) + r, mag = g sum_k |x_k w_k|.
A digit column is an fp32 sum over MMA steps of 64 products; a step adds its products
with at most 7 roundings (or truncations) of 2^-23 of what is summed and one into the
column: 8 K / 64.  Eight columns (7 FMAs), 2 powers of two, 8 splits, the scale and
the bias follow (16 columns, 20 splits at most in these shapes): c = K / 8 + 50.  The magnitudes of the digits of an element add up to
less than 4 of its own (11 / 3 for a 1 above digits of -4).  r: elements of x below
2^-35 (up to 8 rows) or 2^-14 (more) of their row's largest are rounded by 2^-43 or
2^-22 of it, times the weights they meet."""
import numpy as np
import pytest
import torch

import oracle
from oracle import nvfp4_ref as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def lx():
    import video_dit_dynamic_token_b200 as m
    return m


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).to(DEV)


def _weights(lx, rng, N, K, scale=0.05):
    W = _bf16(rng.standard_normal((N, K)) * scale)
    return lx.lx_nvfp4_quantize(W), nv.quant_nvfp4_ref(W.float().cpu().numpy())


def _bound(ref, K, bias=None):
    mag = 4 * ref["mag"] + (0 if bias is None else np.abs(bias)[None, :])
    return 2.0 ** -8 * np.abs(ref["y"]) + (K / 8 + 50) * 2.0 ** -23 * mag + ref["small"] + 1e-38


def _ref(x, wr, bias=None):
    """The oracle's result with the bound r of the rounding of x's small elements."""
    x = np.asarray(x, np.float64)
    ref = oracle.gemv_nvfp4_ref(x, wr, bias)
    M, K = x.shape
    a = np.abs(np.where(np.isfinite(x), x, 0))
    top = a.max(-1, keepdims=True)
    exact, lsb = (-35, -43) if M <= 8 else (-14, -22)
    hit = (a < 2.0 ** exact * top) & (a > 0)
    w = np.abs(oracle.dequant_nvfp4_ref(wr["codes"], wr["sf"], wr["g"]))
    ref["small"] = 2.0 ** lsb * top * (hit.astype(np.float64) @ w.T)
    return ref


def _check(lx, x, wq, wr, bias=None, out=None):
    K = x.shape[1]
    y = lx.lx_nvfp4_gemv(x, wq, None if bias is None else torch.from_numpy(bias).to(DEV), out=out)
    assert lx.lx_last_device_status() == 0
    ref = _ref(x.float().cpu().numpy(), wr, bias)
    off = np.abs(y.float().cpu().numpy() - ref["y"])
    b = _bound(ref, K, bias)
    assert np.all(off <= b), f"{np.max(off / b):.3g} of the bound"
    return y


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(1, 64), (128, 128), (130, 192), (300, 1088), (77, 4672)])
def test_shapes(lx, M, N, K):
    rng = np.random.default_rng(M * 1000 + N + K)
    wq, wr = _weights(lx, rng, N, K)
    bias = rng.standard_normal(N).astype(np.float32) if (M + N) % 2 else None
    _check(lx, _bf16(rng.standard_normal((M, K))), wq, wr, bias)


def test_long_k_in_several_segments(lx):
    """Many turns of the ring in every CTA of a cluster, and an odd number of k-steps."""
    rng = np.random.default_rng(1)
    for M in (1, 16):
        K = 8 * 32 * 128 + 64 * 77
        wq, wr = _weights(lx, rng, 130, K)
        _check(lx, _bf16(rng.standard_normal((M, K))), wq, wr)


def test_exact_sums_bit_exact(lx):
    """Power-of-two scales and small integers make every fp32 sum exact, which pins the
    place of each code, scale and element of x."""
    rng = np.random.default_rng(2)
    N, K = 260, 704
    for M in (1, 5, 16):
        codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
        codes[codes == 8] = 0
        sf = np.array([0x30, 0x38, 0x40, 0x48], np.uint8)[rng.integers(0, 4, (N, K // 16))]
        x = rng.integers(-8, 9, (M, K)).astype(np.float32)
        bias = (rng.integers(-64, 64, N) / 4.0).astype(np.float32)
        wq = lx.NvFp4Tensor(torch.from_numpy(nv.pack_e2m1(codes)).to(DEV), torch.from_numpy(nv.sf_tiled(sf)).to(DEV),
                            torch.tensor([0.5], device=DEV), N, K)
        y = lx.lx_nvfp4_gemv(_bf16(x), wq, torch.from_numpy(bias).to(DEV))
        ref = oracle.gemv_nvfp4_ref(x, {"codes": codes, "sf": sf, "g": np.float32(0.5)}, bias)
        assert np.array_equal(y.float().cpu().numpy(), ref["y_bf16"])


def test_every_code_and_scale(lx):
    """One weight row per (code, scale) pair against a single one in x."""
    codes = np.zeros((127, 64), np.uint8)
    sf = np.zeros((127, 4), np.uint8)
    for s in range(127):
        codes[s, :16] = np.arange(16)
        sf[s, 0] = s
    x = np.zeros((16, 64), np.float32)
    x[np.arange(16), np.arange(16)] = 1
    wq = lx.NvFp4Tensor(torch.from_numpy(nv.pack_e2m1(codes)).to(DEV), torch.from_numpy(nv.sf_tiled(sf)).to(DEV),
                        torch.ones(1, device=DEV), 127, 64)
    y = lx.lx_nvfp4_gemv(_bf16(x), wq)
    want = nv.e2m1_decode(np.arange(16))[:, None] * oracle.e4m3_decode(np.arange(127))[None, :]
    assert np.array_equal(y.float().cpu().numpy(), want)      # 6 significant bits: exact in bf16


def test_wide_range_of_x(lx):
    """Rows of very different size, outliers, zeros, and the smallest and largest values."""
    rng = np.random.default_rng(3)
    N, K = 200, 512
    wq, wr = _weights(lx, rng, N, K, scale=1.0)
    x = rng.standard_normal((12, K))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3] *= np.exp(rng.uniform(-15, 15, K))
    x[4, ::128] = 1e4
    x[5, 1:] = 0
    x[6] *= 1e-38                                     # subnormal bf16
    x[7, 128:] = 0                                    # all-zero chunks
    xb = _bf16(x)
    y = lx.lx_nvfp4_gemv(xb, wq)
    ref = _ref(xb.float().cpu().numpy(), wr)
    # results near the end of fp32's range: subnormal steps of the sums and of bf16
    off = np.abs(y.float().cpu().numpy() - ref["y"])
    assert np.all(off <= _bound(ref, K) + 2.0 ** -133 + K * 2.0 ** -149)
    assert torch.all(y[2] == 0)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_x_stays_in_its_row(lx, bad):
    rng = np.random.default_rng(4)
    wq, wr = _weights(lx, rng, 150, 256)
    x = rng.standard_normal((3, 256))
    clean = _ref(_bf16(x).float().cpu().numpy(), wr)
    x[1, 77] = bad
    y = lx.lx_nvfp4_gemv(_bf16(x), wq).float().cpu().numpy()
    for m in (0, 2):
        assert np.all(np.abs(y[m] - clean["y"][m]) <= _bound(clean, 256)[m])
    want = oracle.gemv_nvfp4_ref(_bf16(x).float().cpu().numpy(), wr)["y"][1]
    assert np.array_equal(np.isnan(y[1]), np.isnan(want))
    assert np.array_equal(y[1][~np.isnan(want)], want[~np.isnan(want)])


def test_strides_and_untouched_padding(lx):
    rng = np.random.default_rng(5)
    N, K = 135, 320
    wq, wr = _weights(lx, rng, N, K)
    big = _bf16(rng.standard_normal((4, K + 128)))
    buf = torch.full((4, N + 6), 5.0, dtype=torch.bfloat16, device=DEV)
    _check(lx, big[:, 64:64 + K], wq, wr, out=buf[:, 3:3 + N])
    assert torch.all(buf[:, :3] == 5.0) and torch.all(buf[:, 3 + N:] == 5.0)


def test_model_projections_sampled(lx):
    """The 14B model's widths: modulation (6 x 5120), output projection, second feed-forward product."""
    for N, K, M in ((30720, 5120, 1), (5120, 5120, 2), (5120, 13824, 16)):
        gen = torch.Generator(device=DEV).manual_seed(N + K)
        W = (torch.randn((N, K), device=DEV, generator=gen) * 0.02).to(torch.bfloat16)
        x = torch.randn((M, K), device=DEV, generator=gen).to(torch.bfloat16)
        wq = lx.lx_nvfp4_quantize(W)
        y = lx.lx_nvfp4_gemv(x, wq)
        rows = np.r_[0, 127, 128, N - 1, np.random.default_rng(N).choice(N, 60, replace=False)]
        wr = nv.quant_nvfp4_ref(W[torch.from_numpy(rows).to(DEV)].float().cpu().numpy(), wq.gscale.item())
        ref = _ref(x.float().cpu().numpy(), wr)
        assert np.all(np.abs(y.float().cpu().numpy()[:, rows] - ref["y"]) <= _bound(ref, K))


def test_equals_the_gemm_on_exact_activations(lx):
    """Activations that NVFP4 holds exactly: the few-row form and the GEMM agree."""
    rng = np.random.default_rng(6)
    N, K, M = 256, 512, 4
    wq, _ = _weights(lx, rng, N, K)
    xc = rng.integers(0, 16, (M, K)).astype(np.uint8)
    xc[xc == 8] = 0
    sf = np.full((M, K // 16), 0x38, np.uint8)
    xq = lx.NvFp4Tensor(torch.from_numpy(nv.pack_e2m1(xc)).to(DEV), torch.from_numpy(nv.sf_tiled(sf)).to(DEV),
                        torch.ones(1, device=DEV), M, K)
    a, b = lx.lx_nvfp4_gemm(xq, wq).float(), lx.lx_nvfp4_gemv(_bf16(nv.e2m1_decode(xc)), wq).float()
    assert lx.lx_last_device_status() == 0
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 1e-3).all()


def test_capture_streams_and_repeatability(lx):
    rng = np.random.default_rng(7)
    wq, wr = _weights(lx, rng, 500, 1024)
    x = _bf16(rng.standard_normal((3, 1024)))
    first = _check(lx, x, wq, wr)
    out = torch.zeros_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lx.lx_nvfp4_gemv(x, wq, out=out)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lx.lx_nvfp4_gemv(x, wq, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    x.copy_(_bf16(rng.standard_normal((3, 1024))))
    g.replay()
    torch.cuda.synchronize()
    ref = _ref(x.float().cpu().numpy(), wr)
    assert np.all(np.abs(out.float().cpu().numpy() - ref["y"]) <= _bound(ref, 1024))


@pytest.mark.parametrize("M,N,K", [(1, 300, 10240), (1, 300, 10304), (8, 300, 1280), (8, 300, 1344), (7, 513, 1408),
                                   (3, 40, 64), (5, 9000, 2048), (2, 6553, 5120), (2, 6554, 5120)])
def test_digits_in_the_product_kernel_and_before_it(lx, M, N, K):
    """Both sides of the rule for where digits are made; then rows that hold infinities and NaN."""
    rng = np.random.default_rng(M + N + K)
    wq, wr = _weights(lx, rng, N, K)
    x = _bf16(rng.standard_normal((M, K)) * 2.0 ** rng.integers(-20, 20, (M, 1)))
    bias = rng.standard_normal(N).astype(np.float32)
    y = _check(lx, x, wq, wr, bias)
    assert (lx.lx_nvfp4_gemv_ws_size(M, N, K) == 0) == (M * K <= 10240 and N * K <= 2 ** 25)
    spoilt = x.clone()
    spoilt[0, K - 1] = float("inf")
    z = lx.lx_nvfp4_gemv(spoilt, wq, torch.from_numpy(bias).to(DEV))
    assert lx.lx_last_device_status() == 0
    w = oracle.dequant_nvfp4_ref(wr["codes"], wr["sf"], wr["g"])[:, K - 1]
    got = z[0].float().cpu().numpy()
    assert np.all(got[w > 0] == np.inf) and np.all(got[w < 0] == -np.inf) and np.all(np.isnan(got[w == 0]))
    assert torch.equal(z[1:], y[1:])


@pytest.mark.parametrize("M", [1, 8, 16])
def test_many_turns_of_the_ring(lx, M):
    """Many stages a CTA, again and again beside copies that hold up the loads: no wait runs out, nothing changes."""
    rng = np.random.default_rng(20 + M)
    N, K = 2700, 30720
    wq, wr = _weights(lx, rng, N, K)
    x = _bf16(rng.standard_normal((M, K)))
    first = _check(lx, x, wq, wr)
    a = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    b, side = torch.empty_like(a), torch.cuda.Stream()
    for _ in range(40):
        with torch.cuda.stream(side):
            b.copy_(a)
        y = lx.lx_nvfp4_gemv(x, wq)
        assert torch.equal(y, first)
    torch.cuda.synchronize()
    assert lx.lx_last_device_status() == 0


def test_one_row_of_any_stride(lx):
    """A single row has no row stride: views whose stride is no multiple of 8, smaller than K or N, or zero."""
    rng = np.random.default_rng(8)
    N, K = 150, 320
    wq, wr = _weights(lx, rng, N, K)
    data = _bf16(rng.standard_normal(K))
    want = _check(lx, data[None], wq, wr)
    buf = torch.zeros(1024, dtype=torch.bfloat16, device=DEV)
    for stride in (0, 1, 321, 325):
        x = torch.as_strided(data, (1, K), (stride, 1))
        out = torch.as_strided(buf, (1, N), (stride, 1))
        buf.zero_()
        assert torch.equal(lx.lx_nvfp4_gemv(x, wq), want)
        lx.lx_nvfp4_gemv(x, wq, out=out)
        assert torch.equal(out, want) and not buf[N:].any()
    assert lx.lx_last_device_status() == 0
