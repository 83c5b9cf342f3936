"""Cases of the token-wise operators over the active voxels of a sparse tensor:
layer normalisation (both directions), rotary positions, and attention within
each batch item (both directions).

Rows are active voxels (or conditioning tokens) in item order; `offsets` are
the int32 [items + 1] row bounds of the items.  With `own` false, `run`
computes an operator in elementary torch operations; with `own` true it calls
the package.
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the tiny random-occupancy set (about 410 voxels): a call whose launch counts
        {"name": "norm_tiny", "op": "norm", "rows": 410, "channels": 16, "type": "f32", "affine": True, "act": "none"},
        # the 512^3 decoder stage: about 1.3 million voxels of 64 channels, norm and SiLU before a conv
        {"name": "norm_decoder", "op": "norm", "rows": 1300007, "channels": 64, "type": "f16", "affine": True, "act": "silu"},
        # training on the 128^3 shells at 128 channels
        {"name": "norm_bwd_shells", "op": "norm_bwd", "rows": 133450, "channels": 128, "type": "bf16", "affine": True, "act": "silu"},
        # training on the 64^3 stage at 512 channels in fp32, an odd row count, no activation
        {"name": "norm_bwd_stage", "op": "norm_bwd", "rows": 20011, "channels": 512, "type": "f32", "affine": True, "act": "none"},
        # queries and keys of a packed qkv projection on the 64^3 stage, voxel coordinates on three axes
        {"name": "rotary_voxels", "op": "rotary", "rows": 20011, "heads": 16, "packed": True, "dim": 64, "axes": 3, "pairs": 10,
         "type": "bf16", "layout": "interleaved", "factor": 1.0, "far": 64, "inverse": False},
        # three new tokens far out on one axis, half of each head, stretched frequencies
        {"name": "rotary_tokens", "op": "rotary", "rows": 3, "heads": 8, "packed": False, "dim": 128, "axes": 1, "pairs": 32,
         "type": "f16", "layout": "half", "factor": 8.0, "far": 1000000, "inverse": False},
        # full self-attention of the 64^3 stage
        {"name": "attn_stage", "op": "attn", "q_rows": "20011", "k_rows": "", "heads": 8, "kv_heads": 8, "dim": 64, "type": "bf16",
         "causal": False, "lse": True},
        # the same stage cut into 8^3 windows of 1 to 512 voxels
        {"name": "attn_windows", "op": "attn", "q_rows": "512*1..512", "k_rows": "", "heads": 8, "kv_heads": 8, "dim": 64, "type": "f16",
         "causal": False, "lse": False},
        # one new token for each item, over a long context with shared heads
        {"name": "attn_tokens", "op": "attn", "q_rows": "8*1..1", "k_rows": "8*1000..32768", "heads": 16, "kv_heads": 4, "dim": 128,
         "type": "bf16", "causal": False, "lse": False},
        # voxels over the conditioning tokens of their item, in fp32; one item has none
        {"name": "attn_cross", "op": "attn", "q_rows": "1500,37,903", "k_rows": "1374,0,700", "heads": 4, "kv_heads": 4, "dim": 64,
         "type": "f32", "causal": False, "lse": True},
        # training on two shells
        {"name": "attn_bwd_shells", "op": "attn_bwd", "q_rows": "9973,8111", "k_rows": "", "heads": 8, "kv_heads": 8, "dim": 64,
         "type": "bf16", "causal": False},
        # training on voxels in sequence, shared heads, wide heads
        {"name": "attn_bwd_causal", "op": "attn_bwd", "q_rows": "6007,130,1", "k_rows": "", "heads": 8, "kv_heads": 2, "dim": 128,
         "type": "f16", "causal": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rotary", "attn", "attn", "attn_bwd", "attn_bwd"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("norm", "norm_bwd"):
        channels = rng.choice([_log(rng, 8, 1024), 16, 64, 128, 192, 256, 512, 1024])
        rows = _log(rng, 1, min(1300000, 30000000 // channels))
        return {"op": op, "rows": rows, "channels": channels, "type": kind, "affine": rng.random() < 0.7,
                "act": rng.choice(["none", "silu", "relu"])}
    if op == "rotary":
        dim = rng.choice([16, 32, 40, 64, 96, 128])
        axes = rng.choice([1, 2, 3])
        pairs = rng.randint(1, dim // 2 // axes)
        return {"op": op, "rows": _log(rng, 1, 130000), "heads": rng.randint(1, 16), "packed": rng.random() < 0.5, "dim": dim, "axes": axes,
                "pairs": pairs, "type": kind, "layout": rng.choice(["interleaved", "half"]), "factor": rng.choice([1.0, 2.0, 8.0]),
                "far": _log(rng, 8, 4000000), "inverse": rng.random() < 0.5}
    kv_heads = rng.choice([1, 2, 3, 4])
    heads = kv_heads * rng.choice([1, 2, 4])
    dim = rng.choice([16, 32, 64, 64, 80, 128, 128])
    form = rng.choice(["self", "windows", "tokens", "cross"]) if op == "attn" else rng.choice(["self", "windows", "cross"])
    most = 3000 if kind == "f32" else 9000
    k_rows = ""
    if form == "self":
        q_rows = ",".join(str(_log(rng, 1 if i else 8, most)) for i in range(rng.randint(1, 3)))
    elif form == "windows":
        q_rows = "%d*1..%d" % (_log(rng, 8, 300), rng.choice([64, 216, 300]))
    elif form == "tokens":
        n = rng.randint(1, 12)
        q_rows, k_rows = "%d*1..1" % n, "%d*1..%d" % (n, _log(rng, 16, 30000))
    else:
        n = rng.randint(1, 4)
        q_rows = ",".join(str(_log(rng, 1, most)) for _ in range(n))
        k_rows = ",".join(str(rng.choice([0, _log(rng, 1, 1500), _log(rng, 1, 1500)]) if i else _log(rng, 8, 1500)) for i in range(n))
    c = {"op": op, "q_rows": q_rows, "k_rows": k_rows, "heads": heads, "kv_heads": kv_heads, "dim": dim, "type": kind,
         "causal": rng.random() < 0.3}
    if op == "attn":
        c["lse"] = rng.random() < 0.5
    return c


def _lengths(text):
    """Rows of each item: "a,b,c", or "n*lo..hi" for n lengths spread over lo..hi."""
    if "*" in text:
        n, span = text.split("*")
        lo, hi = (int(x) for x in span.split(".."))
        r = random.Random(text)
        return [r.randint(lo, hi) for _ in range(int(n))]
    return [int(x) for x in text.split(",")]


def _items(case):
    q = _lengths(case["q_rows"])
    return q, (_lengths(case["k_rows"]) if case["k_rows"] else q)


def _seen(nq, nk, causal):
    """Query-key pairs that an item's attention looks at (causal: the last query sees every key)."""
    if not causal:
        return nq * nk
    first = nk - nq + 1  # keys that query 0 sees
    lo = max(first, 0)
    n = nk - lo + 1 if nk >= lo else 0
    return (lo + nk) * n // 2 if n > 0 else 0


def work(case):
    size = _BYTES[case["type"]]
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, c = case["rows"], case["channels"]
        if op == "norm":
            return {"bytes": 2 * n * c * size + n * 8 + 2 * c * size * case["affine"], "flops": 8 * n * c}
        return {"bytes": 3 * n * c * size + n * 8 + 4 * c * size * case["affine"], "flops": 14 * n * c}
    if op == "rotary":
        n, elems = case["rows"], case["rows"] * case["heads"] * case["dim"]
        return {"bytes": 2 * elems * size + 4 * n * case["axes"], "flops": 6 * n * case["heads"] * case["axes"] * case["pairs"]}
    q, k = _items(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    pairs = sum(_seen(a, b, case["causal"]) for a, b in zip(q, k)) * h
    nq, nk = sum(q), sum(k)
    if op == "attn":
        return {"bytes": (2 * nq * h + 2 * nk * hk) * d * size + 4 * nq * h * case["lse"], "flops": 4 * pairs * d}
    return {"bytes": (4 * nq * h + 4 * nk * hk) * d * size + 4 * nq * h, "flops": 10 * pairs * d}


def _offsets(rows):
    return torch.tensor([0] + torch.tensor(rows).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = _TYPES[case["type"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(kind)

    s = {"case": dict(case)}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, c = case["rows"], case["channels"]
        s["x"] = (torch.randn((n, c), generator=g, device="cuda") * (0.5 + torch.rand((1, c), generator=g, device="cuda"))
                  + 0.3 * torch.randn((1, c), generator=g, device="cuda")).to(kind)
        s["gamma"] = normal(c, scale=0.2, shift=1.0) if case["affine"] else None
        s["beta"] = normal(c, scale=0.2) if case["affine"] else None
        s["eps"] = 1e-5
        if op == "norm_bwd":
            s["dy"] = normal(n, c)
            s["stats"] = _norm_stats(s["x"], s["eps"])
        return s
    if op == "rotary":
        n, h, d = case["rows"], case["heads"], case["dim"]
        if case["packed"]:  # a view of a wider projection's rows
            s["x"] = normal(n, h + (h + 1) // 2, d)[:, :h]
        else:
            s["x"] = normal(n, h, d)
        coords = torch.randint(0, case["far"], (n, 1 + case["axes"]), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = coords[:, 1:]  # (item, position along each axis)
        f = torch.arange(case["pairs"], dtype=torch.float64, device="cuda") / case["pairs"]
        s["freqs"] = (10000.0 ** -f / case["factor"]).expand(case["axes"], -1).contiguous()
        s["scale"] = 1.0 + 0.1 * math.log(case["factor"])
        return s
    q, k = _items(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    s["lengths"] = (q, k)
    s["offsets"], s["k_offsets"] = _offsets(q), _offsets(k)
    s["q"] = normal(sum(q), h, d)
    s["k"], s["v"] = normal(sum(k), hk, d), normal(sum(k), hk, d)
    if op == "attn_bwd":
        s["dout"] = normal(sum(q), h, d)
        s["out"], s["lse"] = _attention(s)
    return s


# ---------------------------------------------------------------- plain forms
def _norm_stats(x, eps):
    x = x.float()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return torch.stack([mean, (var + eps).rsqrt()], 1)


def _act(y, act):
    return y.clamp_min(0) if act == "relu" else y / (1 + torch.exp(-y)) if act == "silu" else y


def _norm(s):
    x, act = s["x"], s["case"]["act"]
    stats = _norm_stats(x, s["eps"])
    y = (x.float() - stats[:, :1]) * stats[:, 1:]
    if s["gamma"] is not None:
        y = y * s["gamma"].float() + s["beta"].float()
    return _act(y, act).to(x.dtype), stats


def _norm_bwd(s):
    x, act, c = s["x"], s["case"]["act"], s["case"]["channels"]
    stats = s["stats"]
    xhat = (x.float() - stats[:, :1]) * stats[:, 1:]
    dy = s["dy"].float()
    affine = s["gamma"] is not None
    gamma = s["gamma"].float() if affine else None
    if act != "none":
        y = xhat * gamma + s["beta"].float() if affine else xhat
        if act == "relu":
            dy = dy * (y > 0)
        else:
            sig = 1 / (1 + torch.exp(-y))
            dy = dy * (sig * (1 + y * (1 - sig)))
    dyg = dy * gamma if affine else dy
    dx = (dyg - dyg.mean(1, keepdim=True) - xhat * (dyg * xhat).mean(1, keepdim=True)) * stats[:, 1:]
    if not affine:
        return dx.to(x.dtype), None, None
    return dx.to(x.dtype), (dy * xhat).sum(0, dtype=torch.float64).to(x.dtype), dy.sum(0, dtype=torch.float64).to(x.dtype)


def _rotary(s):
    x, case = s["x"], s["case"]
    ang = (s["positions"].double()[:, :, None] * s["freqs"]).flatten(1)  # [rows, pairs of all axes]
    cos = (torch.cos(ang) * s["scale"]).float()[:, None]
    sin = (torch.sin(ang) * s["scale"]).float()[:, None]
    if case["inverse"]:
        sin = -sin
    r = ang.shape[1]
    xf = x.float()
    if case["layout"] == "half":
        a, b = xf[..., :r], xf[..., r:2 * r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = xf[..., 0:2 * r:2], xf[..., 1:2 * r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, xf[..., 2 * r:]], -1).to(x.dtype)


def _rows_of(offsets, n):
    """The item and the place in it of each of n rows."""
    rows = torch.arange(n, device="cuda", dtype=torch.int32)
    item = torch.searchsorted(offsets, rows, right=True).long() - 1
    return item, rows.long() - offsets.long()[item]


def _pad(x, offsets, most):
    """[items, heads, most, dim] in 32 bits; places behind an item's rows are zero."""
    rows = offsets.long()[:-1, None] + torch.arange(most, device="cuda")
    there = rows < offsets.long()[1:, None]
    x = torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])
    return x[torch.where(there, rows, x.shape[0] - 1)].transpose(1, 2)


def _scores(s, qp, kp):
    """Scaled scores [items, heads, queries, keys], -inf where a query does not see a key."""
    case, (ql, kl) = s["case"], s["lengths"]
    group = case["heads"] // case["kv_heads"]
    kp = kp.repeat_interleave(group, 1) if group > 1 else kp
    sc = torch.matmul(qp, kp.transpose(2, 3)).mul_(case["dim"] ** -0.5)
    if case["causal"] or min(kl) < max(kl):
        nq = (s["offsets"][1:] - s["offsets"][:-1]).long()[:, None, None]
        nk = (s["k_offsets"][1:] - s["k_offsets"][:-1]).long()[:, None, None]
        i = torch.arange(max(ql), device="cuda")[:, None]
        j = torch.arange(max(kl), device="cuda")
        hidden = j >= nk
        if case["causal"]:
            hidden = hidden | (j > i + nk - nq)
        sc.masked_fill_(hidden[:, None], -math.inf)
    return sc


def _attention(s):
    case, (ql, kl) = s["case"], s["lengths"]
    qp, kp, vp = _pad(s["q"], s["offsets"], max(ql)), _pad(s["k"], s["k_offsets"], max(kl)), _pad(s["v"], s["k_offsets"], max(kl))
    group = case["heads"] // case["kv_heads"]
    sc = _scores(s, qp, kp)
    top = sc.amax(3, keepdim=True)
    p = sc.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, vp.repeat_interleave(group, 1) if group > 1 else vp) / torch.where(total == 0, 1.0, total)
    item, at = _rows_of(s["offsets"], s["q"].shape[0])
    lse = (top + total.log()).squeeze(3)
    return o[item, :, at].to(s["q"].dtype), lse[item, :, at].contiguous()


def _attention_bwd(s):
    case, (ql, kl) = s["case"], s["lengths"]
    group, hk = case["heads"] // case["kv_heads"], case["kv_heads"]
    item, at = _rows_of(s["offsets"], s["q"].shape[0])
    kitem, kat = _rows_of(s["k_offsets"], s["k"].shape[0])
    qp, kp, vp = _pad(s["q"], s["offsets"], max(ql)), _pad(s["k"], s["k_offsets"], max(kl)), _pad(s["v"], s["k_offsets"], max(kl))
    dop = _pad(s["dout"], s["offsets"], max(ql))
    delta = _pad((s["dout"].float() * s["out"].float()).sum(2, keepdim=True), s["offsets"], max(ql))
    lse = torch.where(s["lse"] == -math.inf, 0.0, s["lse"])  # a row that sees nothing: its scores are -inf
    p = _scores(s, qp, kp).sub_(_pad(lse[:, :, None], s["offsets"], max(ql))).exp_()
    wide = lambda t: t.repeat_interleave(group, 1) if group > 1 else t  # noqa: E731
    shared = lambda t: t.unflatten(1, (hk, group)).sum(2) if group > 1 else t  # noqa: E731
    dv = shared(torch.matmul(p.transpose(2, 3), dop))
    ds = torch.matmul(dop, wide(vp).transpose(2, 3)).sub_(delta).mul_(p).mul_(case["dim"] ** -0.5)
    dq = torch.matmul(ds, wide(kp))
    dk = shared(torch.matmul(ds.transpose(2, 3), qp))
    t = s["q"].dtype
    return dq[item, :, at].to(t), dk[kitem, :, kat].to(t), dv[kitem, :, kat].to(t)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own(op, case, state)
    if op == "norm":
        return _norm(state)
    if op == "norm_bwd":
        return _norm_bwd(state)
    if op == "rotary":
        return _rotary(state)
    if op == "attn":
        out, lse = _attention(state)
        return (out, lse) if case["lse"] else (out,)
    return _attention_bwd(state)


def _own(op, case, s):
    import submanifold_sparse_convolution_packed_b200 as smc
    act = None if case.get("act", "none") == "none" else case["act"]
    if op == "norm":
        stats = torch.empty((case["rows"], 2), dtype=torch.float32, device="cuda")
        return smc.layer_norm(s["x"], s["gamma"], s["beta"], eps=s["eps"], act=act, stats=stats), stats
    if op == "norm_bwd":
        return smc.layer_norm_backward(s["dy"], s["x"], s["stats"], s["gamma"], s["beta"], act=act)
    if op == "rotary":
        return smc.rotary(s["x"], s["positions"], s["freqs"], layout=case["layout"], scale=s["scale"], inverse=case["inverse"])
    if op == "attn":
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if case["lse"] else None
        out = smc.attention(s["q"], s["k"], s["v"], s["offsets"], s["k_offsets"], causal=case["causal"], lse=lse)
        return (out, lse) if case["lse"] else (out,)
    return smc.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["offsets"], s["k_offsets"],
                                  causal=case["causal"])


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        x = s["x"].to(torch.float64)
        g = s["gamma"].to(torch.float64) if case["affine"] else torch.ones(1, dtype=torch.float64, device="cuda")
        b = s["beta"].to(torch.float64) if case["affine"] else torch.zeros(1, dtype=torch.float64, device="cuda")
        if op == "norm":
            var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
            rstd = 1 / torch.sqrt(var + s["eps"])
        else:
            mean, rstd = s["stats"].to(torch.float64).split(1, 1)
        xh = (x - mean) * rstd
        z = g * xh + b
        if op == "norm":
            y = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
            return y, torch.cat([mean, rstd], 1)
        dz = s["dy"].to(torch.float64)
        if case["act"] == "relu":
            dz = torch.where(z > 0, dz, 0.0)
        elif case["act"] == "silu":
            sg = torch.sigmoid(z)
            dz = dz * (sg + z * sg * (1 - sg))
        dxh = dz * g
        c = case["channels"]
        dx = rstd / c * (c * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True))
        return (dx, (dz * xh).sum(0), dz.sum(0)) if case["affine"] else (dx, None, None)
    if op == "rotary":
        x = s["x"].to(torch.float64)
        y = x.clone()
        pairs, axes = case["pairs"], case["axes"]
        for j in range(pairs * axes):
            t = s["positions"][:, j // pairs].to(torch.float64) * s["freqs"][j // pairs, j % pairs]
            turn = torch.polar(torch.full_like(t, s["scale"]), -t if case["inverse"] else t)
            i0, i1 = (j, j + pairs * axes) if case["layout"] == "half" else (2 * j, 2 * j + 1)
            z = torch.complex(x[..., i0], x[..., i1]) * turn[:, None]
            y[..., i0], y[..., i1] = z.real, z.imag
        return y
    ql, kl = s["lengths"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = (s[n].to(torch.float64) for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    q0 = k0 = 0
    for nq, nk in zip(ql, kl):
        qs, ks = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        if not nq or not nk:
            continue
        unseen = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(nk - nq + 1) if case["causal"] else None
        for i in range(h):
            c = i // (h // hk)
            a = q[qs, i] @ k[ks, c].T / math.sqrt(d)
            if unseen is not None:
                a.masked_fill_(unseen, -math.inf)
            if op == "attn":
                lse[qs, i] = torch.logsumexp(a, 1)
                out[qs, i] = torch.softmax(a, 1).nan_to_num_(0.0) @ v[ks, c]
                continue
            given = s["lse"][qs, i].to(torch.float64)
            p = torch.exp(a - given.masked_fill(given == -math.inf, 0.0)[:, None])
            do = s["dout"][qs, i].to(torch.float64)
            dv[ks, c] += p.T @ do
            da = p * (do @ v[ks, c].T - (do * s["out"][qs, i].to(torch.float64)).sum(1, keepdim=True)) / math.sqrt(d)
            dq[qs, i] = da @ k[ks, c]
            dk[ks, c] += da.T @ q[qs, i]
    if op == "attn":
        return (out, lse) if case["lse"] else (out,)
    return dq, dk, dv
