"""CPU oracle for attention over packed sequences and behind a shared prefix, and
for the product of few bf16 rows with NVFP4 weights (plain numpy, fp64).

TEST INFRASTRUCTURE ONLY, like ``sparse_attn_ref``; it shares no code with the
CUDA library.

Definitions.  Sequence i owns the query rows [cu_q[i], cu_q[i+1]) and the key
rows [cu_k[i], cu_k[i] + lk), lk = cu_k[i+1] - cu_k[i] or len_k[i].  Row t sees
the keys u < lk, under the causal rule u <= t + lk - lq, and every prefix key:
  o_t = sum_u softmax_u(scale q_t.k_u) v_u,  lse_t = log sum_u exp(scale q_t.k_u),
o = 0 and lse = -inf where nothing is seen.  Query head h reads key/value head
h // (Hq // Hkv).  Hidden keys and values do not enter, whatever they hold.

Pins live in ``tests/test_oracle_packed.py``.
"""
from __future__ import annotations

import numpy as np

from .nvfp4_ref import dequant_nvfp4_ref
from .prologue_ref import bf16_round


def packed_attn_ref(Q, K, V, cu_q, cu_k, causal, scale, len_k=None, Kp=None, Vp=None) -> dict:
    """Q [Hq, Tq, D], K, V [Hkv, Tk, D] (and Kp, Vp [Hkv, Lp, D]).  Returns 'o'
    [Hq, Tq, D], 'lse' [Hq, Tq] (nan in rows of no sequence), and per row what the
    error bounds need: 'absv' [Hq, Tq, D] = sum_u w_u |v_u| and 'smag' [Hq, Tq] =
    max_u scale sum_c |q_c k_c|, 'keys' [Hq, Tq] the number of keys seen."""
    Q, K, V = (np.asarray(x, np.float64) for x in (Q, K, V))
    Hq, Tq, D = Q.shape
    grp = Hq // K.shape[0]
    o = np.full((Hq, Tq, D), np.nan)
    absv = np.full((Hq, Tq, D), np.nan)
    lse, smag, keys = (np.full((Hq, Tq), np.nan) for _ in range(3))
    pre = 0 if Kp is None else np.asarray(Kp).shape[1]
    for i in range(len(cu_q) - 1):
        a, b = int(cu_q[i]), int(cu_q[i + 1])
        c = int(cu_k[i])
        lk = int(cu_k[i + 1]) - c if len_k is None else int(len_k[i])
        for h in range(Hq):
            k, v = K[h // grp, c:c + lk], V[h // grp, c:c + lk]
            if pre:
                k = np.concatenate((np.asarray(Kp, np.float64)[h // grp], k))
                v = np.concatenate((np.asarray(Vp, np.float64)[h // grp], v))
            for t in range(a, b):
                own = max(0, min(lk, t - a + lk - (b - a) + 1)) if causal else lk
                n = pre + own
                keys[h, t] = n
                if n == 0:
                    o[h, t], absv[h, t], lse[h, t], smag[h, t] = 0.0, 0.0, -np.inf, 0.0
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (k[:n] @ Q[h, t])
                    m = s.max()
                    w = np.exp(s - m)
                    o[h, t] = (w @ v[:n]) / w.sum()
                    absv[h, t] = (w @ np.abs(v[:n])) / w.sum()
                    lse[h, t] = m + np.log(w.sum())
                    smag[h, t] = scale * (np.abs(k[:n]) @ np.abs(Q[h, t])).max()
    return {"o": o, "lse": lse, "absv": absv, "smag": smag, "keys": keys}


def packed_attn_bounds(ref, D) -> tuple:
    """(|o| bound, |lse| bound) of a bf16 kernel with fp32 scores and statistics.

    A score is an fp32 sum of D products (error at most 2 D 2^-24 of sum |q k|;
    2 for an adder that truncates), scaled and shifted (3 roundings of values
    up to smag log2 e < 2 smag), and exp2 adds 2^-22: each weight is off by
    eta = 2 D 2^-24 smag + 6 2^-24 smag + 2^-22, and the row sums of n terms
    by 2 n 2^-24 more.  P is rounded to bf16 (2^-8), o too."""
    n, smag = ref["keys"], ref["smag"]
    eta = (2 * D + 6) * 2.0 ** -24 * smag + 2.0 ** -22 + 2 * n * 2.0 ** -24
    bo = 2.0 ** -8 * np.abs(ref["o"]) + (2.0 ** -8 * 1.01 + 2 * eta)[..., None] * ref["absv"] + 1e-30
    bl = eta + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0)) + smag)
    return bo, bl


def gemv_nvfp4_ref(X, wq, bias=None) -> dict:
    """y = X W^T g + bias of bf16 rows X [M, K] and NVFP4 W (dict of quant_nvfp4_ref):
    'y' (exact), 'y_bf16', and 'mag' = g sum_k |x_k w_k|."""
    x = np.asarray(X, np.float64)
    w = dequant_nvfp4_ref(wq["codes"], wq["sf"], 1.0)
    g = np.float64(np.float32(wq["g"]))
    with np.errstate(invalid="ignore"):
        y = (x @ w.T) * g
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[None, :]
    mag = (np.abs(x) @ np.abs(w).T) * g
    return {"y": y, "y_bf16": bf16_round(y), "mag": mag}
