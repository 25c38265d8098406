"""Pins of the packed-attention and few-row NVFP4 oracles against other routes:
torch's fp64 attention, scalar loops, and the plain definition on a dense matrix."""
import math

import numpy as np
import pytest
import torch

import oracle


def _case(seed, lq, lk, hq=4, hkv=2, D=8):
    r = np.random.default_rng(seed)
    cu = lambda v: np.concatenate(([0], np.cumsum(v)))
    return (r.standard_normal((hq, sum(lq), D)), r.standard_normal((hkv, sum(lk), D)),
            r.standard_normal((hkv, sum(lk), D)), cu(lq), cu(lk))


@pytest.mark.parametrize("causal", [False, True])
def test_matches_torch_attention_per_sequence(causal):
    lq, lk = [3, 1, 7, 5], [5, 4, 7, 9]
    Q, K, V, cq, ck = _case(0, lq, lk)
    ref = oracle.packed_attn_ref(Q, K, V, cq, ck, causal, 0.3)
    for i, (a, b) in enumerate(zip(lq, lk)):
        q = torch.from_numpy(Q[:, cq[i]:cq[i + 1]])
        k, v = (torch.from_numpy(x[:, ck[i]:ck[i + 1]]).repeat_interleave(2, 0) for x in (K, V))
        mask = torch.ones(a, b, dtype=torch.bool).tril(b - a) if causal else None
        want = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=mask, scale=0.3)
        assert np.abs(ref["o"][:, cq[i]:cq[i + 1]] - want.numpy()).max() < 1e-12
        s = (q @ k.transpose(1, 2)) * 0.3
        if causal:
            s = s.masked_fill(~mask, -math.inf)
        assert np.abs(ref["lse"][:, cq[i]:cq[i + 1]] - torch.logsumexp(s, -1).numpy()).max() < 1e-12


def test_scalar_loops_with_rows_that_see_nothing():
    lq, lk = [4, 2, 0, 1], [2, 0, 3, 1]          # rows before the first key; no keys; no rows
    Q, K, V, cq, ck = _case(1, lq, lk, hq=2, hkv=1, D=4)
    ref = oracle.packed_attn_ref(Q, K, V, cq, ck, True, 0.5)
    for h in range(2):
        for i in range(4):
            for t in range(lq[i]):
                see = [u for u in range(lk[i]) if u <= t + lk[i] - lq[i]]
                row = cq[i] + t
                if not see:
                    assert np.all(ref["o"][h, row] == 0) and ref["lse"][h, row] == -np.inf
                    continue
                w = [math.exp(0.5 * sum(Q[h, row, c] * K[0, ck[i] + u, c] for c in range(4))) for u in see]
                for c in range(4):
                    want = sum(x * V[0, ck[i] + u, c] for x, u in zip(w, see)) / sum(w)
                    assert abs(ref["o"][h, row, c] - want) < 1e-12
                assert abs(ref["lse"][h, row] - math.log(sum(w))) < 1e-12


def test_prefix_is_concatenation_and_len_k_cuts():
    lq, lk, Lp = [2, 3], [4, 3], 6
    Q, K, V, cq, ck = _case(2, lq, lk, D=8)
    r = np.random.default_rng(3)
    Kp, Vp = r.standard_normal((2, Lp, 8)), r.standard_normal((2, Lp, 8))
    got = oracle.packed_attn_ref(Q, K, V, cq, ck, True, 0.4, Kp=Kp, Vp=Vp)
    cat = lambda P, X: np.concatenate([np.concatenate((P, X[:, ck[i]:ck[i + 1]]), 1) for i in range(2)], 1)
    ck2 = np.concatenate(([0], np.cumsum([Lp + n for n in lk])))
    want = oracle.packed_attn_ref(Q, cat(Kp, K), cat(Vp, V), cq, ck2, True, 0.4)
    assert np.abs(got["o"] - want["o"]).max() < 1e-13 and np.abs(got["lse"] - want["lse"]).max() < 1e-13
    cut = oracle.packed_attn_ref(Q, K, V, cq, ck, False, 0.4, len_k=[3, 1])
    keep = np.r_[0:3, 4:5]
    same = oracle.packed_attn_ref(Q, K[:, keep], V[:, keep], cq, [0, 3, 4], False, 0.4)
    assert np.array_equal(cut["o"], same["o"])


def test_hidden_values_do_not_enter():
    Q, K, V, cq, ck = _case(4, [3], [3], hq=1, hkv=1)
    clean = oracle.packed_attn_ref(Q, K, V, cq, ck, True, 1.0)
    K[0, 2], V[0, 2] = np.nan, np.inf
    got = oracle.packed_attn_ref(Q, K, V, cq, ck, True, 1.0)
    assert np.array_equal(got["o"][0, :2], clean["o"][0, :2]) and not np.isfinite(got["o"][0, 2]).all()


def test_gemv_against_scalar_loops():
    r = np.random.default_rng(5)
    W, X = r.standard_normal((5, 64)).astype(np.float32), r.standard_normal((2, 64)).astype(np.float32)
    wq = oracle.quant_nvfp4_ref(W)
    bias = r.standard_normal(5).astype(np.float32)
    y = oracle.gemv_nvfp4_ref(X, wq, bias)["y"]
    mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for m in range(2):
        for n in range(5):
            acc = 0.0
            for k in range(64):
                c, s = int(wq["codes"][n, k]), int(wq["sf"][n, k // 16])
                e, f = s >> 3, s & 7
                sv = (f / 8 * 2.0 ** -6) if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
                acc += float(X[m, k]) * mags[c & 7] * (-1 if c & 8 else 1) * sv
            assert abs(y[m, n] - (acc * float(wq["g"]) + float(bias[n]))) < 1e-9
