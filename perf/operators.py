"""Cases of the serving operators: packed attention, attention behind a shared prefix, and
products of few rows with NVFP4 weights.

Each case runs in the plain form (elementary torch operations in fp32) or, where ``own`` is
true, through the library's entry points; ``exact`` computes the definition in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
# (query heads, key/value heads, head dimension): the video model's 40 heads of 128, the small
# test shape of 2 heads of 64, and grouped forms with power-of-two and odd group sizes
HEADS = [(40, 40, 128), (40, 8, 128), (40, 10, 128), (2, 2, 64), (2, 1, 64), (16, 16, 64), (28, 4, 128),
         (32, 8, 128), (12, 2, 64), (9, 3, 128), (24, 1, 128)]


def listed():
    p = {"op": "packed", "causal": True, "same": True, "cache": False, "spare": 0, "lens": 1}
    x = {"op": "prefix", "causal": True, "spare": 0, "lens": 2}
    g = {"op": "gemv"}
    return [
        # three very short prompts: nothing but latency
        dict(p, name="packed_tiny", n=3, q_lo=5, q_hi=77, k_lo=5, k_hi=77, heads=2, kv_heads=1, dim=64),
        # a batch of prompts of uneven length with grouped heads, some rows of the buffer unused
        dict(p, name="packed_prompts", n=24, q_lo=17, q_hi=2000, k_lo=17, k_hi=2000, heads=40, kv_heads=8, dim=128,
             spare=37),
        # frame-causal video: the whole 480p token grid as one sequence, the model's 40 heads of 128
        dict(p, name="packed_480p", n=1, q_lo=32760, q_hi=32760, k_lo=32760, k_hi=32760, heads=40, kv_heads=40,
             dim=128),
        # cross-attention of video tokens to two text prompts
        dict(p, name="packed_cross", n=2, q_lo=7000, q_hi=9000, k_lo=77, k_hi=512, heads=40, kv_heads=40, dim=128,
             causal=False, same=False),
        # one new token per sequence over caches of uneven fill
        dict(p, name="packed_decode", n=48, q_lo=1, q_hi=1, k_lo=200, k_hi=8000, heads=40, kv_heads=8, dim=128,
             same=False, cache=True),
        # four continuations of a short common prompt
        dict(x, name="prefix_tiny", n=4, q_lo=1, q_hi=1, k_lo=1, k_hi=20, prefix=200, heads=2, kv_heads=2, dim=64),
        # 64 continuations of one long prompt, one token each
        dict(x, name="prefix_decode", n=64, q_lo=1, q_hi=1, k_lo=1, k_hi=500, prefix=8192, heads=40, kv_heads=8,
             dim=128),
        # a 720p token grid kept as the prefix, 16 short chunks behind it
        dict(x, name="prefix_720p", n=16, q_lo=1, q_hi=9, k_lo=9, k_hi=300, prefix=75600, heads=40, kv_heads=8,
             dim=128),
        # a small projection of one row
        dict(g, name="gemv_small", m=1, n=256, k=512, bias=True),
        # the six modulation vectors of one timestep
        dict(g, name="gemv_modulation", m=1, n=30720, k=5120, bias=True),
        # an attention output projection for a guided pair
        dict(g, name="gemv_pair", m=2, n=5120, k=5120, bias=True),
        # the second feed-forward projection for 16 rows
        dict(g, name="gemv_ffn16", m=16, n=5120, k=13824, bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "cross", "decode", "prefix", "prefix", "gemv", "gemv"])
    if kind == "gemv":
        return {"op": "gemv", "m": rng.randint(1, 16), "n": _log(rng, 100, 30720), "k": 64 * _log(rng, 8, 216),
                "bias": rng.random() < 0.5}
    while True:
        hq, hkv, d = rng.choice(HEADS)
        c = {"op": "prefix" if kind == "prefix" else "packed", "heads": hq, "kv_heads": hkv, "dim": d, "causal": True,
             "spare": rng.choice([0, 0, rng.randint(1, 200)]), "lens": rng.randint(1, 1 << 20)}
        if kind == "prompt":
            hi = _log(rng, 64, 32760)
            lo = _log(rng, 1, hi)
            c.update(n=_log(rng, 1, 200), q_lo=lo, q_hi=hi, k_lo=lo, k_hi=hi, same=True, cache=False,
                     causal=rng.random() < 0.8)
        elif kind == "cross":
            hi, khi = _log(rng, 64, 20000), _log(rng, 16, 2000)
            c.update(n=_log(rng, 1, 8), q_lo=_log(rng, 1, hi), q_hi=hi, k_lo=_log(rng, 1, khi), k_hi=khi, same=False,
                     cache=False, causal=False)
        elif kind == "decode":
            khi, q = _log(rng, 64, 60000), rng.choice([1, 1, 1, 2, 4])
            c.update(n=_log(rng, 1, 200), q_lo=1, q_hi=q, k_lo=_log(rng, q, khi), k_hi=khi, same=False,
                     cache=rng.random() < 0.5)
        else:
            khi, q = _log(rng, 8, 2000), rng.choice([1, 1, 1, 3, 9])
            c.update(n=_log(rng, 1, 200), q_lo=1, q_hi=q, k_lo=_log(rng, q, max(q, khi)), k_hi=max(q, khi),
                     prefix=_log(rng, 64, 75600))
        keys = c["k_hi"] + c.get("prefix", 0)
        pairs = float(c["n"]) * c["q_hi"] * keys * hq * d
        scores = float(c["n"]) * c["q_hi"] * keys * (hq // hkv)
        held = float(c["n"]) * max(c["k_hi"] * hkv, c["q_hi"] * hq) * d
        if pairs <= 2e12 and scores <= 3e9 and held <= 1.2e9:
            return c


# ---------------------------------------------------------------- lengths and work
def _lengths(case):
    """(query lengths, key lengths) of the case's sequences, from the case alone."""
    r = random.Random(case["lens"])
    lq = [_log(r, case["q_lo"], case["q_hi"]) for _ in range(case["n"])]
    if case.get("same"):
        return lq, list(lq)
    return lq, [max(a if case["causal"] else 1, _log(r, case["k_lo"], case["k_hi"])) for a in lq]


def work(case):
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k / 2 + n * k / 16 + 2 * m * (n + k) + 4 * n * case["bias"], "flops": 2 * m * n * k}
    lq, lk = _lengths(case)
    h, hk, d, pre = case["heads"], case["kv_heads"], case["dim"], case.get("prefix", 0)
    pairs = 0
    for a, b in zip(lq, lk):
        # causal, aligned at the end: query t sees b - a + t + 1 keys
        pairs += a * pre + (a * (b - a) + a * (a + 1) // 2 if case["causal"] else a * b)
    rows, keys = sum(lq), sum(lk) + pre
    return {"bytes": 4 * rows * h * d + 4 * rows * h + 4 * keys * hk * d, "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + salt)


def _cumulative(lens):
    out = [0]
    for v in lens:
        out.append(out[-1] + v)
    return out


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tokens(rows, heads, dim, gen, scale=1.0):
    """A bf16 [1, heads, rows, dim] view of a token-major buffer, as projections leave it."""
    t = torch.randn((rows, heads, dim), device=DEV, generator=gen) * scale
    return t.to(torch.bfloat16).transpose(0, 1).unsqueeze(0)


def _e2m1_values():
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)


def _nvfp4_weights(n, k, gen):
    """NVFP4 codes, tiled scales and global scale of random weights, in the library's layouts."""
    w = torch.randn((n, k), device=DEV, generator=gen) * 0.02
    g = w.abs().max() / 2688
    s = (w.view(n, k // 16, 16).abs().amax(-1) / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn)
    sg = s.float() * g
    y = w.view(n, k // 16, 16) / torch.where(sg > 0, sg, torch.ones_like(sg)).unsqueeze(-1)
    mag = torch.bucketize(y.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV))
    code = (mag + 8 * ((y < 0) & (mag > 0))).view(n, k).to(torch.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    tiles = -(-n // 128)
    sb = torch.zeros((tiles * 128, k // 16), dtype=torch.uint8, device=DEV)
    sb[:n] = s.view(torch.uint8)
    # row r = 128 t + 32 c + l, block j = 4 ks + jj  ->  [t, ks, l, c, jj]
    sf = sb.view(tiles, 4, 32, k // 64, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes.contiguous(), sf, g.reshape(1).float()


def prepare(case, seed):
    gen = _gen(seed, 17)
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        codes, sf, g = _nvfp4_weights(n, k, gen)
        x = torch.randn((m, k), device=DEV, generator=gen).to(torch.bfloat16)
        bias = torch.randn(n, device=DEV, generator=gen) if case["bias"] else None
        return {"case": case, "x": x, "codes": codes, "sf": sf, "g": g, "bias": bias}
    lq, lk = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    rows = sum(lq) + case["spare"]
    held = [case["k_hi"]] * case["n"] if case.get("cache") else lk  # a cache keeps a slot of full length for each
    s = {"case": case, "max_q": max(lq), "max_k": max(lk),
         "q": _tokens(rows, h, d, gen, 1.5), "k": _tokens(sum(held), hk, d, gen), "v": _tokens(sum(held), hk, d, gen),
         "cu_q": _i32(_cumulative(lq)), "cu_k": _i32(_cumulative(held)),
         "len_k": _i32(lk) if case.get("cache") else None,
         "out": torch.zeros((rows, h, d), dtype=torch.bfloat16, device=DEV).transpose(0, 1).unsqueeze(0),
         "lse": torch.zeros((h, rows), dtype=torch.float32, device=DEV)}
    if case["op"] == "prefix":
        s["kp"] = _tokens(case["prefix"], hk, d, gen)
        s["vp"] = _tokens(case["prefix"], hk, d, gen)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attention(s):
    """Padded batches, a slab of key/value heads at a time: products, mask, exponentials, sums in fp32."""
    c = s["case"]
    n, mq, mk, hk, d = c["n"], s["max_q"], s["max_k"], c["kv_heads"], c["dim"]
    grp = c["heads"] // hk
    rows = s["q"].shape[2]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq = cq[1:] - cq[:-1]
    lk = s["len_k"].long() if s["len_k"] is not None else ck[1:] - ck[:-1]
    tq, tk = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    iq, ik = cq[:-1, None] + tq, ck[:-1, None] + tk
    live_q, live_k = tq < lq[:, None], tk < lk[:, None]
    seen = live_k[:, None, :].expand(n, mq, mk)
    if c["causal"]:
        seen = seen & (tk <= (tq + (lk - lq)[:, None])[:, :, None])
    seen = seen[:, None]  # [n, 1, mq, mk]
    iq_in, ik_in = iq.clamp(max=rows - 1), ik.clamp(max=s["k"].shape[2] - 1)
    put = torch.where(live_q, iq, rows)  # rows of the padding go to a row of their own
    out = torch.zeros((c["heads"], rows + 1, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((c["heads"], rows + 1), device=DEV)
    slab = max(1, min(hk, int(1.5e9 // (grp * n * mq * (mk + c.get("prefix", 0))))))
    for h in range(0, hk, slab):
        e = min(hk, h + slab)
        q = s["q"][0, h * grp:e * grp].float()[:, iq_in]  # [(e-h) grp, n, mq, d]
        q = q.view(e - h, grp, n, mq, d).transpose(1, 2) / math.sqrt(d)  # [e-h, n, grp, mq, d]
        k = s["k"][0, h:e].float()[:, ik_in]
        v = s["v"][0, h:e].float()[:, ik_in]
        sc = (q.reshape(e - h, n, grp * mq, d) @ k.transpose(-1, -2)).view(e - h, n, grp, mq, mk)
        sc = sc.masked_fill(~seen, -math.inf)
        top = sc.amax(-1, keepdim=True)
        if c["op"] == "prefix":
            kp, vp = s["kp"][0, h:e].float(), s["vp"][0, h:e].float()
            sp = (q.reshape(e - h, n * grp * mq, d) @ kp.transpose(-1, -2)).view(e - h, n, grp, mq, -1)
            top = torch.maximum(top, sp.amax(-1, keepdim=True))
        at = torch.where(top == -math.inf, torch.zeros_like(top), top)
        sc = torch.exp(sc.sub_(at))
        total = sc.sum(-1, keepdim=True)
        o = (sc.view(e - h, n, grp * mq, mk) @ v).view(e - h, n, grp, mq, d)
        if c["op"] == "prefix":
            sp = torch.exp(sp.sub_(at))
            total = total + sp.sum(-1, keepdim=True)
            o = o + (sp.view(e - h, n * grp * mq, -1) @ vp).view(e - h, n, grp, mq, d)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        ls = (top + torch.log(total)).squeeze(-1)
        heads = slice(h * grp, e * grp)
        out[heads, put] = o.transpose(1, 2).reshape((e - h) * grp, n, mq, d).to(torch.bfloat16)
        lse[heads, put] = ls.transpose(1, 2).reshape((e - h) * grp, n, mq)
    return {"o": out[:, :rows].unsqueeze(0), "lse": lse[:, :rows]}


def _plain_gemv(s):
    n, k = s["codes"].shape[0], s["codes"].shape[1] * 2
    code = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(n, k)
    w = _e2m1_values()[code.long()]
    tiles = -(-n // 128)
    sb = s["sf"].view(tiles, k // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles * 128, k // 16)[:n]
    w = w.view(n, k // 16, 16) * sb.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    y = (s["x"].float() @ w.view(n, k).t()) * s["g"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(torch.bfloat16)}


def run(state):
    case = state["case"]
    if not own:
        return _plain_gemv(state) if case["op"] == "gemv" else _plain_attention(state)
    import video_dit_dynamic_token_b200 as lx
    if case["op"] == "gemv":
        w = lx.NvFp4Tensor(state["codes"], state["sf"], state["g"], case["n"], case["k"])
        return {"y": lx.lx_nvfp4_gemv(state["x"], w, state["bias"])}
    a = {"causal": case["causal"], "len_k": state["len_k"], "out": state["out"], "lse": state["lse"]}
    if case["op"] == "packed":
        o = lx.lx_attn_packed(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], **a)
    else:
        o = lx.lx_attn_prefix(state["q"], state["kp"], state["vp"], state["k"], state["v"], state["cu_q"],
                              state["cu_k"], **a)
    return {"o": o, "lse": state["lse"]}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        y = torch.empty((m, n), dtype=torch.float64, device=DEV)
        x = s["x"].double()
        for t in range(0, n, 128):  # the scales are laid out in tiles of 128 rows
            rows = min(128, n - t)
            w = torch.empty((rows, k), dtype=torch.float64, device=DEV)
            for half, shift in ((0, 0), (1, 4)):
                c = (s["codes"][t:t + rows] >> shift) & 15
                w[:, half::2] = mags[(c & 7).long()] * (1.0 - 2.0 * (c >> 3).double())
            r = torch.arange(rows, device=DEV)[:, None]
            j = torch.arange(k // 16, device=DEV)[None, :]
            at = ((t // 128) * (k // 64) + j // 4) * 512 + (r % 32) * 16 + (r // 32) * 4 + j % 4
            w = w.view(rows, k // 16, 16) * s["sf"][at].view(torch.float8_e4m3fn).double()[:, :, None]
            y[:, t:t + rows] = x @ w.view(rows, k).t()
        y = y * s["g"].double()
        if s["bias"] is not None:
            y = y + s["bias"].double()
        return {"y": y}
    lq, lk = _lengths(case)
    h, grp, d = case["heads"], case["heads"] // case["kv_heads"], case["dim"]
    q, k, v = (s[x][0].double() for x in ("q", "k", "v"))
    out = torch.zeros((1, h, q.shape[1], d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((h, q.shape[1]), dtype=torch.float64, device=DEV)
    cu_q, cu_k = _cumulative(lq), s["cu_k"].tolist()
    for i, (a, b) in enumerate(zip(lq, lk)):
        for j in range(h):
            keys, vals = k[j // grp, cu_k[i]:cu_k[i] + b], v[j // grp, cu_k[i]:cu_k[i] + b]
            front = 0
            if case["op"] == "prefix":
                front = case["prefix"]
                keys = torch.cat((s["kp"][0, j // grp].double(), keys))
                vals = torch.cat((s["vp"][0, j // grp].double(), vals))
            for r in range(0, a, 4096):
                z = min(a, r + 4096)
                last = front + b if not case["causal"] else front + b - a + z  # keys that any of these rows sees
                logit = (q[j, cu_q[i] + r:cu_q[i] + z] @ keys[:last].t()) * (d ** -0.5)
                if case["causal"]:
                    edge = front + b - a + torch.arange(r, z, device=DEV)
                    logit[torch.arange(last, device=DEV)[None, :] > edge[:, None]] = -math.inf
                norm = torch.logsumexp(logit, -1)
                out[0, j, cu_q[i] + r:cu_q[i] + z] = torch.exp(logit - norm[:, None]) @ vals[:last]
                lse[j, cu_q[i] + r:cu_q[i] + z] = norm
    return {"o": out, "lse": lse}
