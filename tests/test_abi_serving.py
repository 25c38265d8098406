"""Host-side refusals of the packed-attention, prefix and few-row NVFP4 entry points
(no GPU: every call is rejected before anything is launched)."""
import ctypes

import pytest

from video_dit_dynamic_token_b200 import _abi, build

INV, UNS, ALI, WSP = _abi.LX_ERR_INVALID, _abi.LX_ERR_UNSUPPORTED, _abi.LX_ERR_ALIGN, _abi.LX_ERR_WORKSPACE
S = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def _view(ptr=0x10000, B=1, H=8, L=1000, D=128, sL=None, sH=None):
    sL = H * D if sL is None else sL
    return _abi.LxBhld(ptr, B, H, L, D, L * sL, D if sH is None else sH, sL)


def _pack(cq=0x1000, ck=0x2000, used=None, n=4):
    return _abi.LxPack(cq, ck, used, n)


def _packed(lib, q=None, k=None, v=None, pk=None, scale=0.1, o=None, lse=None, ws=0x100000, wb=1 << 40):
    q = _view() if q is None else q
    k = _view(H=2) if k is None else k
    v, o = k if v is None else v, q if o is None else o
    pk = _pack() if pk is None else pk
    r = ctypes.byref
    return lib.lx_attn_packed(r(q), r(k), r(v), r(pk), 1, scale, r(o), lse, ws, wb, S)


def test_packed_refusals(lib):
    assert _packed(lib, q=_view(H=7)) == INV                      # not a multiple of the key/value heads
    assert _packed(lib, q=_view(B=2)) == INV
    assert _packed(lib, k=_view(H=2, D=64)) == INV                # head dimensions differ
    assert _packed(lib, v=_view(H=2, L=999)) == INV
    assert _packed(lib, o=_view(L=999)) == INV
    assert _packed(lib, q=_view(D=96), k=_view(H=2, D=96)) == UNS
    assert _packed(lib, q=_view(H=258), k=_view(H=2)) == UNS      # more than 128 query heads a key/value head
    assert _packed(lib, q=_view(ptr=0x10008)) == ALI
    assert _packed(lib, k=_view(H=2, sL=260)) == ALI
    assert _packed(lib, q=_view(L=0)) == INV
    for bad in (_pack(cq=None), _pack(ck=None), _pack(n=0), _pack(n=-3)):
        assert _packed(lib, pk=bad) == INV
    assert _packed(lib, pk=_pack(n=(1 << 30) + 1)) == UNS
    for bad in (_pack(cq=0x1002), _pack(ck=0x2001), _pack(used=0x3003)):
        assert _packed(lib, pk=bad) == ALI
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert _packed(lib, scale=bad) == INV
    assert _packed(lib, lse=0x5002) == ALI
    long = _view(H=2, L=3000)                                     # enough keys to split
    assert _packed(lib, k=long, ws=None) == WSP
    assert _packed(lib, k=long, ws=0x100010) == ALI
    r = ctypes.byref
    q, k, pk = _view(), _view(H=2), _pack()
    assert lib.lx_attn_packed(None, r(k), r(k), r(pk), 1, 0.1, r(q), None, 0x100000, 1 << 40, S) == INV
    assert lib.lx_attn_packed(r(q), r(k), r(k), None, 1, 0.1, r(q), None, 0x100000, 1 << 40, S) == INV


def test_workspace_sizes(lib):
    r, n = ctypes.byref, ctypes.c_size_t()
    q, k = _view(L=4), _view(H=2)
    assert lib.lx_attn_packed_ws_size(r(q), r(k), 4, r(n)) == 0
    splits, rows = 128, 4 * 8
    assert n.value == 256 + splits * rows * 8 + splits * rows * 128 * 4
    assert _packed(lib, q=q, k=k, wb=n.value - 1) == WSP
    # many rows: a bounded workspace, at least two splits
    big = _view(L=30000)
    assert lib.lx_attn_prefix_ws_size(r(big), r(n)) == 0
    assert 2 * 30000 * 8 * (128 * 4 + 8) <= n.value <= 2 * 30000 * 8 * (128 * 4 + 8) + 1024
    mid = _view(L=1000)
    assert lib.lx_attn_prefix_ws_size(r(mid), r(n)) == 0 and n.value <= (64 << 20) + 1024
    # prompts that fill the GPU need none
    assert lib.lx_attn_packed_ws_size(r(_view(H=40, L=8000)), r(_view(H=40, L=8000)), 4, r(n)) == 0 and n.value == 0
    assert lib.lx_attn_packed_ws_size(r(q), r(k), 0, r(n)) == INV
    assert lib.lx_attn_packed_ws_size(r(q), r(k), 4, None) == INV
    assert lib.lx_attn_prefix_ws_size(r(q), None) == INV


def test_prefix_refusals(lib):
    r = ctypes.byref
    q, k, pk = _view(), _view(H=2), _pack()
    call = lambda kp, vp=None, wb=1 << 40, ws=0x100000: lib.lx_attn_prefix(
        r(q), r(kp), r(kp if vp is None else vp), r(k), r(k), r(pk), 1, 0.1, r(q), None, ws, wb, S)
    assert call(_view(H=4, L=50)) == INV
    assert call(_view(H=2, L=50, D=64)) == INV
    assert call(_view(H=2, L=50), _view(H=2, L=51)) == INV
    assert call(_view(H=2, L=50, B=2)) == INV
    assert call(_view(H=2, L=50, ptr=0x20004)) == ALI
    assert call(_view(H=2, L=50), wb=100) == WSP
    assert call(_view(H=2, L=50), ws=None) == WSP


def test_gemv_refusals(lib):
    x, c, f, g, y = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
    call = lambda x=x, M=1, ldx=256, c=c, f=f, g=g, b=None, N=100, K=256, y=y, ldy=100, ws=0x70000, wb=1 << 40: \
        lib.lx_nvfp4_gemv(x, M, ldx, c, f, g, b, N, K, y, ldy, ws, wb, S)
    for k in ("x", "c", "f", "g", "y"):
        assert call(**{k: None}) == INV
    assert call(M=0) == INV and call(N=0) == INV and call(K=0) == INV
    assert call(K=96, ldx=96) == INV
    assert call(ldx=248) == INV and call(ldy=99) == INV
    assert call(M=17) == UNS
    assert call(N=1 << 31, ldy=1 << 31) == UNS
    assert call(ldx=260) == ALI
    assert call(x=x + 2) == ALI and call(c=c + 8) == ALI and call(f=f + 8) == ALI
    assert call(g=g + 2) == ALI and call(b=0x60002) == ALI and call(y=y + 1) == ALI
    assert call(K=(1 << 24) + 64, ldx=(1 << 24) + 64) == UNS
    n = ctypes.c_size_t()
    size = lambda M, K, N=100: lib.lx_nvfp4_gemv_ws_size(M, N, K, ctypes.byref(n))
    assert size(3, 320) == 0 and n.value == 0 and size(8, 1280) == 0 and n.value == 0   # digits in the product kernel
    assert size(2, 5120, 6553) == 0 and n.value == 0 and size(2, 5120, 6554) == 0 and n.value == 2 * 16 * 2560 + 256
    assert size(8, 1344) == 0 and n.value == 8 * 16 * 672 + 256      # 16 digits for up to 8 rows
    big = dict(M=8, K=1344, ldx=1344)
    assert call(**big, wb=n.value - 1) == WSP and call(**big, ws=None) == WSP and call(**big, ws=0x70010) == ALI
    assert size(9, 320) == 0 and n.value == 9 * 8 * 160 + 256        # 11520 is a multiple of 256
    assert size(17, 320) == UNS and size(1, (1 << 24) + 64) == UNS and size(1, 64, (1 << 30) + 1) == UNS
    assert size(1, 100) == INV and size(0, 64) == INV and size(1, 64, 0) == INV
    assert lib.lx_nvfp4_gemv_ws_size(1, 64, 64, None) == INV


def test_the_workspace_does_not_grow_with_the_rows(lib):
    """Partial rows are kept for sequences that are split, in 64 MB at most: 200 prompts of 77 tokens."""
    r, n = ctypes.byref, ctypes.c_size_t()
    for rows, heads, seqs in ((77 * 24, 40, 24), (77 * 200, 40, 200), (100000, 40, 100000), (1 << 20, 64, 1 << 20)):
        q = _view(H=heads, L=rows)
        assert lib.lx_attn_packed_ws_size(r(q), r(q), seqs, r(n)) == 0
        assert 0 < n.value <= (64 << 20) + 4 * seqs + 1024
        pk = _pack(n=seqs)
        assert _packed(lib, q=q, k=q, pk=pk, wb=n.value - 1) == WSP
    # few rows: 128 splits of each, as many as a call can have, and a word for each sequence
    q, k = _view(L=100), _view(H=2)
    assert lib.lx_attn_packed_ws_size(r(q), r(k), 100, r(n)) == 0
    assert n.value == 512 + 128 * 800 * (8 + 512)


def test_more_keys_than_rows_leave_the_split_to_the_lengths(lib):
    """Prompts that fill the GPU need no workspace, unless a long cache may be among them."""
    r, n = ctypes.byref, ctypes.c_size_t()
    for keys, some in ((2112, False), (2112 + 2048, False), (2112 + 2049, True), (125000, True)):
        q, k = _view(H=40, L=2112), _view(H=8, L=keys)
        assert lib.lx_attn_packed_ws_size(r(q), r(k), 68, r(n)) == 0
        assert (n.value > 0) == some


def test_a_scale_whose_exponent_overflows(lib):
    """scale * log2(e), which the kernels work with, has to be finite: 0 * inf would be NaN."""
    assert _packed(lib, scale=2.4e38) == INV and _packed(lib, scale=3.4e38) == INV
    assert _packed(lib, scale=2.3e38, k=_view(H=2, L=3000), ws=None) == WSP       # the check after it
