"""Attention over packed sequences and behind a shared prefix (lx_attn_packed,
lx_attn_prefix) against the fp64 oracle.  The bounds are packed_attn_bounds of
oracle/packed_ref.py, derived there from the roundings the kernels make."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def lx():
    import video_dit_dynamic_token_b200 as m
    return m


def _i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def _cu(lens, start=0):
    out = [start]
    for v in lens:
        out.append(out[-1] + v)
    return out


def _rows(gen, H, T, D, scale=1.0, token_major=True):
    if token_major:
        t = (torch.randn((T, H, D), generator=gen) * scale).to(torch.bfloat16).to(DEV)
        return t.transpose(0, 1).unsqueeze(0)
    return (torch.randn((1, H, T, D), generator=gen) * scale).to(torch.bfloat16).to(DEV)


def _np(t):
    return t[0].float().cpu().numpy()


def _check(got, lse, ref, D, rows=None):
    o, l = got[0].float().cpu().numpy(), lse.cpu().numpy()
    live = ~np.isnan(ref["keys"])
    if rows is not None:
        live &= rows
    bo, bl = oracle.packed_attn_bounds(ref, D)
    fin = live[..., None] & np.isfinite(ref["o"])
    assert np.isfinite(o[fin]).all()
    off = np.abs(o - np.where(fin, ref["o"], o))
    assert np.all(off[fin] <= bo[fin]), f"o: {np.max(off[fin] / bo[fin]):.3g} of the bound"
    none = live & np.isneginf(ref["lse"])
    assert np.all(l[none] == -np.inf)
    ok = live & np.isfinite(ref["lse"])
    d = np.abs(l[ok] - ref["lse"][ok])
    assert np.all(d <= bl[ok]), f"lse: {np.max(d / bl[ok]):.3g} of the bound"


def _run(lx, lq, lk, hq, hkv, D, causal, seed=0, token_major=True, scale=None, used=None, spare=0, first=0, qs=1.5,
         prefix=0, ref=True):
    gen = torch.Generator().manual_seed(seed)
    Tq, Tk = first + sum(lq) + spare, sum(lk) + spare
    Q = _rows(gen, hq, max(Tq, 1), D, qs, token_major)
    K, V = (_rows(gen, hkv, max(Tk, 1), D, 1.0, token_major) for _ in range(2))
    cq, ck = _cu(lq, first), _cu(lk)
    out = torch.full_like(Q, 7.0)
    lse = torch.full((hq, Q.shape[2]), 9.0, device=DEV)
    lk_t = None if used is None else _i32(used)
    Kp = Vp = None
    if prefix:
        Kp, Vp = (_rows(gen, hkv, prefix, D, 1.0, token_major) for _ in range(2))
        lx.lx_attn_prefix(Q, Kp, Vp, K, V, _i32(cq), _i32(ck), causal=causal, scale=scale, len_k=lk_t, out=out, lse=lse)
    else:
        lx.lx_attn_packed(Q, K, V, _i32(cq), _i32(ck), causal=causal, scale=scale, len_k=lk_t, out=out, lse=lse)
    assert lx.lx_last_device_status() == 0
    # rows of no sequence are left as they were
    for a, b in ((0, first), (cq[-1], Q.shape[2])):
        assert torch.all(out[:, :, a:b] == 7.0) and torch.all(lse[:, a:b] == 9.0)
    if not ref:
        return Q, K, V, out, lse
    r = oracle.packed_attn_ref(_np(Q), _np(K), _np(V), cq, ck, causal, D ** -0.5 if scale is None else scale, used,
                               None if Kp is None else _np(Kp), None if Vp is None else _np(Vp))
    _check(out, lse, r, D)
    return Q, K, V, out, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_one_sequence_one_tile(lx, D, causal):
    _run(lx, [1], [1], 1, 1, D, causal)
    _run(lx, [5], [5], 2, 1, D, causal)
    _run(lx, [100], [128], 1, 1, D, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,D", [(2, 2, 64), (4, 2, 128), (5, 1, 128), (6, 2, 64), (9, 3, 128), (24, 1, 64)])
def test_ragged_lengths(lx, hq, hkv, D, causal):
    _run(lx, [1, 17, 64, 130, 3], [1, 17, 64, 130, 3], hq, hkv, D, causal, seed=3)


@pytest.mark.parametrize("D", [64, 128])
def test_empty_sequences_and_rows_that_see_nothing(lx, D):
    # no rows; no keys; more rows than keys under the causal rule (the first rows see nothing)
    _run(lx, [3, 0, 4, 130, 0, 2], [3, 5, 0, 2, 0, 200], 2, 1, D, True, seed=4, spare=3, first=2)
    _run(lx, [3, 0, 4, 130, 0, 2], [3, 5, 0, 2, 0, 200], 2, 1, D, False, seed=4, spare=3, first=2)


@pytest.mark.parametrize("lk", [1, 127, 128, 129, 255, 257, 700])
def test_single_token_over_keys(lx, lk):
    _run(lx, [1, 1, 1], [lk, 1, 3 * lk], 4, 2, 128, True, seed=lk)


def test_cache_slots_partly_used(lx):
    _run(lx, [1, 2, 1, 3], [300, 300, 300, 300], 8, 2, 64, True, seed=6, used=[1, 300, 0, 129])


def test_scale_and_layout(lx):
    _run(lx, [40, 70], [90, 70], 4, 4, 128, True, seed=7, token_major=False, scale=0.02)
    _run(lx, [40, 70], [90, 70], 4, 4, 64, True, seed=8, scale=1.0, qs=0.3)


def test_large_scores_rescale_the_accumulator(lx):
    """Keys that grow along the sequence make the running maximum jump at every tile."""
    gen = torch.Generator().manual_seed(9)
    D, n = 128, 900
    Q = _rows(gen, 2, n, D)
    K, V = _rows(gen, 1, n, D), _rows(gen, 1, n, D)
    K = (K.float() * torch.linspace(0.1, 12, n, device=DEV)[None, None, :, None]).to(torch.bfloat16)
    for causal in (True, False):
        lse = torch.empty((2, n), device=DEV)
        o = lx.lx_attn_packed(Q, K, V, _i32([0, n]), _i32([0, n]), causal=causal, lse=lse)
        assert lx.lx_last_device_status() == 0
        _check(o, lse, oracle.packed_attn_ref(_np(Q), _np(K), _np(V), [0, n], [0, n], causal, D ** -0.5), D)


@pytest.mark.parametrize("hq,hkv,D", [(40, 40, 128), (40, 8, 128), (32, 8, 64)])
def test_prompts_that_fill_the_gpu(lx, hq, hkv, D):
    """Several items for every SM; checked on sampled heads."""
    lq = [700, 33, 1500, 257]
    Q, K, V, out, lse = _run(lx, lq, lq, hq, hkv, D, True, seed=10, spare=5, ref=False)
    cu = _cu(lq)
    for h in (0, hq // 2 + 1, hq - 1):
        g = h // (hq // hkv)
        r = oracle.packed_attn_ref(_np(Q)[h:h + 1], _np(K)[g:g + 1], _np(V)[g:g + 1], cu, cu, True, D ** -0.5)
        _check(out[:, h:h + 1], lse[h:h + 1], r, D)


def test_alone_and_in_a_large_pack(lx):
    """The same sequences by themselves and in a pack."""
    D, hq, hkv = 128, 40, 40
    lq = [400, 900, 130] * 4
    Q, K, V, out, lse = _run(lx, lq, lq, hq, hkv, D, True, seed=11, ref=False)
    assert lx.lx_attn_packed_ws_size(Q, K, len(lq)) == 0
    cu = _cu(lq)
    for i in (0, 1, 2, 11):
        a, b = cu[i], cu[i + 1]
        l1 = torch.empty((hq, b - a), device=DEV)
        o1 = lx.lx_attn_packed(Q[:, :, a:b], K[:, :, a:b], V[:, :, a:b], _i32([0, b - a]), _i32([0, b - a]), lse=l1)
        assert lx.lx_last_device_status() == 0
        assert (o1 - out[:, :, a:b]).abs().max() <= 0.02
        assert (l1 - lse[:, a:b]).abs().max() <= 1e-4


# ---------------------------------------------------------------- values in masked places
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("lq", [[60, 150], [1, 1]])
def test_what_hidden_rows_hold_does_not_enter(lx, bad, lq):
    """Rows behind each sequence's keys in use, and past the last sequence."""
    gen = torch.Generator().manual_seed(12)
    D, used, cap = 128, [150, 201], 256
    Q, K, V = _rows(gen, 2, sum(lq) + 4, D), _rows(gen, 1, 2 * cap + 9, D), _rows(gen, 1, 2 * cap + 9, D)
    cq, ck = _cu(lq), [0, cap, 2 * cap]
    ref = oracle.packed_attn_ref(_np(Q), _np(K), _np(V), cq, ck, True, D ** -0.5, used)
    for i in range(2):
        K[:, :, ck[i] + used[i]:ck[i + 1]] = bad
        V[:, :, ck[i] + used[i]:ck[i + 1]] = bad
    K[:, :, 2 * cap:] = bad
    V[:, :, 2 * cap:] = bad
    Q[:, :, cq[-1]:] = bad
    lse = torch.zeros((2, Q.shape[2]), device=DEV)
    o = lx.lx_attn_packed(Q, K, V, _i32(cq), _i32(ck), len_k=_i32(used), lse=lse)
    assert lx.lx_last_device_status() == 0
    _check(o, lse, ref, D)


@pytest.mark.parametrize("n", [90, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_keys_hidden_by_the_causal_rule_do_not_enter(lx, n, bad):
    """A non-finite key and value reach the rows that see them and no other."""
    gen = torch.Generator().manual_seed(13)
    D = 64
    Q, K, V = _rows(gen, 2, n, D), _rows(gen, 1, n, D), _rows(gen, 1, n, D)
    at = n - 25
    ref = oracle.packed_attn_ref(_np(Q), _np(K), _np(V), [0, n], [0, n], True, D ** -0.5)
    K[:, :, at] = bad
    V[:, :, at] = bad
    lse = torch.empty((2, n), device=DEV)
    o = lx.lx_attn_packed(Q, K, V, _i32([0, n]), _i32([0, n]), lse=lse)
    assert lx.lx_last_device_status() == 0
    rows = np.zeros((2, n), bool)
    rows[:, :at] = True
    _check(o, lse, ref, D, rows)
    assert torch.isnan(o[:, :, at:].float()).all()


def test_finite_value_behind_a_non_finite_one(lx):
    """V alone non-finite and visible: inf where its weight is not zero."""
    gen = torch.Generator().manual_seed(14)
    n, D = 140, 128
    Q, K, V = _rows(gen, 1, n, D), _rows(gen, 1, n, D), _rows(gen, 1, n, D)
    V[0, 0, 50, 3] = float("inf")
    o = lx.lx_attn_packed(Q, K, V, _i32([0, n]), _i32([0, n]))
    assert lx.lx_last_device_status() == 0
    assert torch.isfinite(o[0, 0, :50].float()).all()
    assert torch.isinf(o[0, 0, 50:, 3].float()).all() and (o[0, 0, 50:, 3] > 0).all()
    keep = [c for c in range(D) if c != 3]
    assert torch.isfinite(o[0, 0, 50:][:, keep].float()).all()


# ---------------------------------------------------------------- prefix
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,D", [(2, 2, 64), (5, 1, 128), (8, 2, 128)])
def test_prefix(lx, hq, hkv, D, causal):
    _run(lx, [1, 1, 1, 1], [1, 20, 0, 7], hq, hkv, D, causal, seed=20, prefix=200, spare=3)
    _run(lx, [9, 1, 40, 0, 3], [9, 300, 40, 6, 0], hq, hkv, D, causal, seed=21, prefix=129, first=1)
    _run(lx, [1], [1], hq, hkv, D, causal, seed=22, prefix=1)


def test_prefix_equals_packed_concatenation(lx):
    gen = torch.Generator().manual_seed(23)
    hq, hkv, D, Lp = 10, 2, 128, 1000
    lq, lk = [1, 4, 33], [60, 4, 200]
    Q = _rows(gen, hq, sum(lq), D)
    K, V, Kp, Vp = (_rows(gen, hkv, t, D) for t in (sum(lk), sum(lk), Lp, Lp))
    ck = _cu(lk)
    cat = lambda P, X: torch.cat([torch.cat((P, X[:, :, ck[i]:ck[i + 1]]), 2) for i in range(3)], 2).contiguous()
    a = lx.lx_attn_prefix(Q, Kp, Vp, K, V, _i32(_cu(lq)), _i32(ck))
    b = lx.lx_attn_packed(Q, cat(Kp, K), cat(Vp, V), _i32(_cu(lq)), _i32(_cu([Lp + n for n in lk])))
    assert lx.lx_last_device_status() == 0
    assert (a.float() - b.float()).abs().max() <= 0.02


# ---------------------------------------------------------------- calls
def test_many_sequences(lx):
    """More sequences than threads of a block, some empty."""
    r = np.random.default_rng(30)
    lk = r.integers(0, 60, 700).tolist()
    lq = [min(1, k) for k in lk]
    _run(lx, lq, lk, 2, 1, 64, True, seed=31)
    _run(lx, lq, lk, 2, 1, 64, True, seed=32, prefix=77)
    lq = r.integers(0, 40, 700).tolist()
    Q, K, V, out, lse = _run(lx, lq, lq, 16, 16, 64, True, seed=33, ref=False)
    cu = _cu(lq)
    rr = oracle.packed_attn_ref(_np(Q)[5:6], _np(K)[5:6], _np(V)[5:6], cu, cu, True, 64 ** -0.5)
    _check(out[:, 5:6], lse[5:6], rr, 64)


def test_malformed_lengths_are_reported_and_left_out(lx):
    from video_dit_dynamic_token_b200._abi import LX_ERR_PLAN
    gen = torch.Generator().manual_seed(34)
    Q, K, V = (_rows(gen, 2, 100, 64) for _ in range(3))
    good = torch.full_like(Q, 3.0)
    for cq, ck, used in (([0, 50, 40, 100], [0, 50, 60, 100], None), ([0, 50, 80, 101], [0, 50, 60, 100], None),
                         ([0, 50, 60, 100], [0, 50, -4, 100], None), ([0, 50, 60, 100], [0, 50, 60, 100], [50, 11, 41]),
                         ([0, 50, 60, 100], [0, 50, 60, 100], [50, 10, -1])):
        o = good.clone()
        lx.lx_attn_packed(Q, K, V, _i32(cq), _i32(ck), len_k=None if used is None else _i32(used), out=o)
        assert lx.lx_last_device_status() == LX_ERR_PLAN
        assert torch.isfinite(o.float()).all() and not torch.all(o[:, :, :50] == 3.0)
        o = good.clone()
        lx.lx_attn_prefix(Q, K, V, K, V, _i32(cq), _i32(ck), len_k=None if used is None else _i32(used), out=o)
        assert lx.lx_last_device_status() == LX_ERR_PLAN
    assert lx.lx_last_device_status() == 0


def test_captured_call_follows_the_lengths(lx):
    gen = torch.Generator().manual_seed(35)
    D, n, cap = 128, 3, 400
    Q, K, V = _rows(gen, 4, n, D), _rows(gen, 2, n * cap, D), _rows(gen, 2, n * cap, D)
    cq, ck, used = _i32(range(n + 1)), _i32([0, cap, 2 * cap, 3 * cap]), _i32([1, 1, 1])
    out, lse = torch.zeros_like(Q), torch.zeros((4, n), device=DEV)
    ws = torch.empty(lx.lx_attn_packed_ws_size(Q, K, n), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    call = lambda: lx.lx_attn_packed(Q, K, V, cq, ck, len_k=used, out=out, lse=lse, ws=ws)
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for lens in ([1, 1, 1], [400, 17, 128], [3, 0, 399]):
        used.copy_(torch.tensor(lens, dtype=torch.int32))
        K.copy_(torch.randn(K.shape, generator=gen).to(torch.bfloat16))
        ws.fill_(255)
        g.replay()
        assert lx.lx_last_device_status() == 0
        _check(out, lse, oracle.packed_attn_ref(_np(Q), _np(K), _np(V), range(n + 1), ck.tolist(), True, D ** -0.5,
                                                lens), D)


def test_two_streams_and_repeatability(lx):
    gen = torch.Generator().manual_seed(36)
    lq = [3, 200, 77]
    Q, K, V = (_rows(gen, 4, 280, 64) for _ in range(3))
    cu = _i32(_cu(lq))
    first = lx.lx_attn_packed(Q, K, V, cu, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(lx.lx_attn_packed(Q, K, V, cu, cu))
    torch.cuda.synchronize()
    assert lx.lx_last_device_status() == 0
    for o in outs:
        assert torch.equal(o[:, :, :280], first[:, :, :280])


def test_rows_far_into_a_long_cache(lx):
    """Offsets past 2^31 elements: keys of a sequence that lies behind 8.4 M rows."""
    D, T = 128, 2 ** 23 + 4000
    K = torch.zeros((1, 2, T, D), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros((1, 2, T, D), dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator().manual_seed(37)
    a, n = T - 1000, 700
    K[:, :, a:a + n] = _rows(gen, 2, n, D)
    V[:, :, a:a + n] = _rows(gen, 2, n, D)
    Q = _rows(gen, 4, 3, D)
    lse = torch.empty((4, 3), device=DEV)
    o = lx.lx_attn_packed(Q, K, V, _i32([0, 3]), _i32([a, a + n]), lse=lse)
    assert lx.lx_last_device_status() == 0
    _check(o, lse, oracle.packed_attn_ref(_np(Q), _np(K[:, :, a:a + n]), _np(V[:, :, a:a + n]), [0, 3], [0, n], True,
                                          D ** -0.5), D)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,prefix", [(6, 6, 0), (5, 5, 0), (10, 2, 0), (9, 3, 0), (12, 4, 700), (15, 3, 700), (4, 1, 700)])
def test_rests_of_one_row_tile(lx, hq, hkv, prefix, causal):
    """Sequences that end in a single row tile, with even and odd numbers of key/value heads, split and whole."""
    tq = 128 // (hq // hkv)
    lens = [2 * tq + 1, 3 * tq, 2 * tq + tq // 2, tq, tq + 1, 4 * tq]
    _run(lx, lens, [n + 300 for n in lens], hq, hkv, 64, causal, seed=hq + prefix, prefix=prefix, spare=3)


@pytest.mark.parametrize("pad", [8, 16])
def test_rows_of_the_output_at_16_and_32_bytes(lx, pad):
    gen = torch.Generator().manual_seed(38)
    lq = [130, 1, 40]
    Q, K, V = (_rows(gen, 4, 171, 64, token_major=False) for _ in range(3))
    cu = _cu(lq)
    room = torch.full((1, 4, 171, 64 + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    for first in (0, pad):
        out, lse = room[..., first:first + 64], torch.empty((4, 171), device=DEV)
        lx.lx_attn_packed(Q, K, V, _i32(cu), _i32(cu), out=out, lse=lse)
        assert lx.lx_last_device_status() == 0
        _check(out, lse, oracle.packed_attn_ref(_np(Q), _np(K), _np(V), cu, cu, True, 64 ** -0.5), 64)
        rest = torch.cat((room[..., :first], room[..., first + 64:]), -1)
        assert torch.all(rest == 7.0)
        room.fill_(7.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,D,lq,lk", [(1, 1, 64, [2700], [2700]), (2, 2, 128, [2500], [2500]), (8, 2, 64, [700, 3, 40], [3100, 300, 40]),
                                            (6, 2, 128, [300], [4000])])
def test_few_long_prompts_are_split(lx, hq, hkv, D, lq, lk, causal):
    """Too few row tiles for the SMs: the keys of full row tiles are split and joined."""
    Q, K, V, out, lse = _run(lx, lq, lk, hq, hkv, D, causal, seed=sum(lk), spare=2, ref=False)
    assert lx.lx_attn_packed_ws_size(Q, K, len(lq)) > 0
    cq, ck = _cu(lq), _cu(lk)
    rows = np.zeros((hq, cq[-1] + 2), bool)
    for a, b in zip(cq, cq[1:]):   # every 37th row and the last of each sequence
        rows[:, a:b:37] = rows[:, b - 1] = True
    keep = np.flatnonzero(rows[0])
    for h in (0, hq - 1):
        g = h // (hq // hkv)
        for i in range(len(lq)):
            for t in keep[(keep >= cq[i]) & (keep < cq[i + 1])]:
                n = lk[i] - lq[i] + (t - cq[i]) + 1 if causal else lk[i]
                r = oracle.packed_attn_ref(_np(Q)[h:h + 1, t:t + 1], _np(K)[g:g + 1, ck[i]:ck[i] + n],
                                           _np(V)[g:g + 1, ck[i]:ck[i] + n], [0, 1], [0, n], False, D ** -0.5)
                _check(out[:, h:h + 1, t:t + 1], lse[h:h + 1, t:t + 1], r, D)


# ---------------------------------------------------------------- rows computed again, in splits and for long
def _hidden(lx, lq, lk, hq, hkv, D, bad, at, seed, prefix=0, key_too=True):
    """A non-finite key and value at key `at` of the last sequence: rows that do not see it, and those that do."""
    gen = torch.Generator().manual_seed(seed)
    Q, K, V = _rows(gen, hq, sum(lq), D), _rows(gen, hkv, sum(lk), D), _rows(gen, hkv, sum(lk), D)
    pre = [_rows(gen, hkv, prefix, D) for _ in range(2)] if prefix else []
    cq, ck = _cu(lq), _cu(lk)
    ref = oracle.packed_attn_ref(_np(Q), _np(K), _np(V), cq, ck, True, D ** -0.5, None, *[_np(t) for t in pre])
    if key_too:
        K[:, :, ck[-2] + at] = bad
    V[:, :, ck[-2] + at] = bad
    lse = torch.empty((hq, sum(lq)), device=DEV)
    if prefix:
        o = lx.lx_attn_prefix(Q, *pre, K, V, _i32(cq), _i32(ck), lse=lse)
    else:
        assert lx.lx_attn_packed_ws_size(Q, K, len(lq)) > 0
        o = lx.lx_attn_packed(Q, K, V, _i32(cq), _i32(ck), lse=lse)
    assert lx.lx_last_device_status() == 0
    rows = np.ones((hq, sum(lq)), bool)
    first = cq[-2] + max(0, at - (lk[-1] - lq[-1]))     # the first row that sees the key
    rows[:, first:] = False
    _check(o, lse, ref, D, rows)
    if first < cq[-1]:
        spoilt = o[:, :, first:].float()
        if key_too or bad != bad:
            assert torch.isnan(spoilt).all()
        else:
            assert (spoilt == bad).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("key_too", [True, False])
@pytest.mark.parametrize("hq,hkv,D,lq,lk", [(2, 1, 64, [3, 9], [50, 5000]), (4, 2, 128, [9], [3000]),
                                            (3, 1, 128, [2, 7], [300, 2600]), (6, 6, 64, [1, 40], [700, 4100])])
def test_hidden_keys_do_not_enter_splits(lx, hq, hkv, D, lq, lk, bad, key_too):
    """A few tokens over a cache whose keys are split: the key before the last one, and one in the middle of the rows."""
    for back in (1, lq[-1] // 2):
        _hidden(lx, lq, lk, hq, hkv, D, bad, lk[-1] - 1 - back, 40 + back, key_too=key_too)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,D", [(1, 1, 64), (2, 2, 128)])
def test_hidden_keys_do_not_enter_split_prompts(lx, hq, hkv, D, bad):
    n = 2300
    _hidden(lx, [n], [n], hq, hkv, D, bad, n - 30, 43, key_too=False)
    _hidden(lx, [n], [n], hq, hkv, D, bad, 1200, 44)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,D", [(2, 1, 64), (8, 2, 128), (3, 3, 128)])
def test_hidden_keys_do_not_enter_behind_a_prefix(lx, hq, hkv, D, bad):
    for key_too in (True, False):
        _hidden(lx, [1, 9], [30, 9], hq, hkv, D, bad, 6, 45, prefix=300, key_too=key_too)
        _hidden(lx, [4, 40], [4, 900], hq, hkv, D, bad, 870, 46, prefix=1500, key_too=key_too)


def test_rows_computed_again_for_longer_than_a_wait(lx):
    """A million tokens with a last value that is not finite: 127 rows are computed again, which takes a warp
    longer than the 2 s that any wait of the others is limited to."""
    n, D = 1 << 20, 64
    gen = torch.Generator(device=DEV).manual_seed(47)
    Q, K, V = (torch.randn((1, 1, n, D), device=DEV, generator=gen).to(torch.bfloat16) for _ in range(3))
    V[:, :, n - 1] = float("inf")
    lse = torch.empty((1, n), device=DEV)
    cu = _i32([0, n])
    assert lx.lx_attn_packed_ws_size(Q, K, 1) == 0
    o = lx.lx_attn_packed(Q, K, V, cu, cu, lse=lse)
    assert lx.lx_last_device_status() == 0
    assert torch.isfinite(o[0, 0, :n - 1].float()).all() and (o[0, 0, n - 1] == float("inf")).all()
    k, v = _np(K), _np(V)
    for t in (n - 2, n - 65, n - 128, n - 129, n // 2):
        r = oracle.packed_attn_ref(_np(Q)[:, t:t + 1], k[:, :t + 1], v[:, :t + 1], [0, 1], [0, t + 1], True, D ** -0.5)
        _check(o[:, :, t:t + 1], lse[:, t:t + 1], r, D)


# ---------------------------------------------------------------- room for partial rows
def _check_sampled(lx, lq, lk, hq, hkv, D, seqs, seed, heads=None, spare=3):
    """A call whose K and V are made on the GPU, checked on whole sequences of some heads."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    mk = lambda T, H, f: ((torch.randn((T, H, D), device=DEV, generator=gen) * f).to(torch.bfloat16)
                          .transpose(0, 1).unsqueeze(0))
    cq, ck = _cu(lq), _cu(lk)
    Q, K, V = mk(cq[-1] + spare, hq, 1.5), mk(ck[-1], hkv, 1.0), mk(ck[-1], hkv, 1.0)
    out, lse = torch.full_like(Q, 7.0), torch.full((hq, Q.shape[2]), 9.0, device=DEV)
    ws = torch.full((max(lx.lx_attn_packed_ws_size(Q, K, len(lq)), 256) + 256,), 255, dtype=torch.uint8, device=DEV)
    lx.lx_attn_packed(Q, K, V, _i32(cq), _i32(ck), out=out, lse=lse, ws=ws[:-256])
    assert lx.lx_last_device_status() == 0
    assert torch.all(ws[-256:] == 255)
    assert torch.all(out[:, :, cq[-1]:] == 7.0) and torch.all(lse[:, cq[-1]:] == 9.0)
    for i in seqs:
        a, b, c, d = cq[i], cq[i + 1], ck[i], ck[i + 1]
        for h in (0, hq - 1) if heads is None else heads:
            g = h // (hq // hkv)
            r = oracle.packed_attn_ref(_np(Q[:, h:h + 1, a:b]), _np(K[:, g:g + 1, c:d]), _np(V[:, g:g + 1, c:d]),
                                       [0, b - a], [0, d - c], True, D ** -0.5)
            _check(out[:, h:h + 1, a:b], lse[h:h + 1, a:b], r, D)
    return Q, K


def test_many_short_prompts_need_little_room(lx):
    """Prompts of at most a row tile each: nothing is split, and the workspace does not grow with the rows."""
    Q, K = _check_sampled(lx, [77] * 200, [77] * 200, 40, 40, 128, (0, 99, 199), 50)
    assert lx.lx_attn_packed_ws_size(Q, K, 200) <= (64 << 20) + 4096
    _check_sampled(lx, [40, 77, 1, 128, 16] * 20, [40, 77, 1, 128, 16] * 20, 9, 3, 64, (0, 1, 2, 3, 99), 51)


def test_splits_that_do_not_fit_get_longer(lx):
    """More rows with splits than the workspace holds: 80 sequences of 32 tokens over 1,300 keys, eight over 2,600."""
    lk = [2600 if i % 11 == 3 else 1300 for i in range(80)]
    _check_sampled(lx, [32] * 80, lk, 32, 8, 128, (0, 3, 14, 79), 52)


def test_heads_without_a_neighbour_are_not_split_where_there_is_no_room(lx):
    """One key/value head, whose narrow items split their keys between two streams, and too many rows for that."""
    lk = [130 + 7 * (i % 10) for i in range(2700)]
    _check_sampled(lx, [1] * 2700, lk, 24, 1, 128, (0, 1, 1350, 2699), 53)
    _check_sampled(lx, [1] * 700, lk[:700], 24, 1, 128, (0, 1, 350, 699), 54)


def test_split_sequences_among_many(lx):
    """A few long sequences among hundreds of short ones: each finds its own partial rows."""
    r = np.random.default_rng(55)
    lq = r.integers(0, 4, 900).tolist()
    lk = r.integers(3, 60, 900).tolist()
    long = (0, 5, 6, 130, 131, 501, 898, 899)
    for i in long:
        lq[i], lk[i] = 1 + i % 3, 2000 + 13 * i
    _check_sampled(lx, lq, lk, 4, 2, 64, long + (1, 7, 132, 897), 56)
    _check_sampled(lx, lq, lk, 6, 3, 64, long + (1, 7, 132, 897), 57)


@pytest.mark.parametrize("hq,hkv,D", [(40, 8, 128), (9, 3, 64)])
def test_a_long_cache_among_prompts_is_split(lx, hq, hkv, D):
    """Prompts that fill the GPU with single tokens in one call, one of them over a long cache."""
    lq, lk = [500, 1, 700, 1, 1, 900] + [1] * 20, [500, 400, 700, 24000, 1, 900] + [300] * 20
    if hkv == 3:
        lq[2] = lk[2] = 5000
    _check_sampled(lx, lq, lk, hq, hkv, D, (1, 3, 4, 25), 58, heads=(0, hq - 1))
    _check_sampled(lx, lq, lk, hq, hkv, D, (0,), 58, heads=(1,))


@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("hq,hkv,rows", [(4, 2, 8), (4, 2, 300), (3, 1, 40)])
def test_a_table_that_counts_rows_again_and_again(lx, hq, hkv, rows, prefix):
    """cu_q goes up and down: half the sequences own the same rows, with keys that would be split."""
    from video_dit_dynamic_token_b200._abi import LX_ERR_PLAN
    n, D, cap = 600, 64, 3000
    gen = torch.Generator().manual_seed(59)
    Q, K, V = _rows(gen, hq, rows + 4, D), _rows(gen, hkv, cap, D), _rows(gen, hkv, cap, D)
    out, lse = torch.full_like(Q, 7.0), torch.full((hq, rows + 4), 9.0, device=DEV)
    cq = _i32([0 if i % 2 == 0 else rows for i in range(n + 1)])
    ck = _i32([0] + [cap] * n)
    used = _i32([cap] + [0] * (n - 1))
    for keys, lens in ((ck, None), (ck, used), (_i32([0 if i % 2 == 0 else cap for i in range(n + 1)]), None)):
        a = (Q, K[:, :, :prefix], V[:, :, :prefix], K, V) if prefix else (Q, K, V)
        call = lx.lx_attn_prefix if prefix else lx.lx_attn_packed
        call(*a, cq, keys, len_k=lens, out=out, lse=lse)
        assert lx.lx_last_device_status() == LX_ERR_PLAN
        assert torch.all(out[:, :, rows:] == 7.0) and torch.all(lse[:, rows:] == 9.0)
    good = lx.lx_attn_packed(Q, K, V, _i32([0, rows]), _i32([0, cap]))
    assert lx.lx_last_device_status() == 0 and torch.isfinite(good[:, :, :rows].float()).all()
