"""Layer norm, rotary positions and attention on the GPU against plain 64-bit
forms.  Tolerances count roundings: u = eps / 2 of the type relative to the
value for its one rounding, and multiples of 2^-24 of the magnitudes that enter
for the fp32 arithmetic before it."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import submanifold_sparse_convolution_packed_b200 as smc

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    smc.lib()
    yield
    smc.set_alloc_fail_after(0)


def u_of(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def close(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - ref).abs()[bad].max()),
                                 float(tol.expand_as(ref)[bad].min()))


# ------------------------------------------------------------------ layer norm
def norm_ref(x, gamma, beta, eps, act, stats=None):
    x = x.double()
    if stats is None:
        mean = x.mean(1, keepdim=True)
        rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    else:
        mean, rstd = stats.double().split(1, 1)
    xh = (x - mean) * rstd
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    z = g * xh + b
    y = z.clamp_min(0) if act == "relu" else z * torch.sigmoid(z) if act == "silu" else z
    # x and the mean are off by a few fp32 ulp of |x| + |mean| before the product with rstd
    err = 64 * E * (torch.as_tensor(g).abs() * ((x.abs() + mean.abs()) * rstd + xh.abs()) + torch.as_tensor(b).abs())
    return y, z, xh, mean, rstd, err + 16 * E * (4 + z.abs()) * y.abs()


NORM_SHAPES = [(1, 1), (7, 3), (410, 16), (33, 64), (5, 65), (129, 100), (1001, 128), (64, 130), (3, 257), (40, 512),
               (17, 500), (9, 1000), (30, 1024), (6, 1025), (5, 5000), (20011, 64), (70000, 8)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n, c", NORM_SHAPES)
@pytest.mark.parametrize("act, affine", [(None, True), ("silu", True), ("relu", False)])
def test_layer_norm(n, c, dtype, act, affine):
    g = gen(n * 1000 + c)
    x = normal(g, n, c, dtype=dtype, scale=2.0, shift=1.5)
    gamma = normal(g, c, dtype=dtype, scale=0.3, shift=1.0) if affine else None
    beta = normal(g, c, dtype=dtype, scale=0.3) if affine else None
    stats = torch.empty(n, 2, device="cuda")
    y = smc.layer_norm(x, gamma, beta, eps=1e-5, act=act, stats=stats)
    ref, _, _, mean, rstd, err = norm_ref(x, gamma, beta, 1e-5, act)
    close(y, ref, u_of(dtype) * ref.abs() + err + 1e-7 * (dtype == F16), "y")
    close(stats[:, :1], mean, 16 * E * x.double().abs().mean(1, keepdim=True), "mean")
    # the variance is off by a few ulp of itself and by (error of the mean)^2
    close(stats[:, 1:], rstd, 64 * E * rstd * (1 + (mean * rstd) ** 2 * E), "rstd")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n, c", [(1, 8), (7, 9), (410, 16), (33, 64), (129, 100), (1001, 128), (64, 130), (9, 1000),
                                  (30, 1024), (6, 1025), (5, 5000), (200, 2048), (20011, 64), (70000, 8)])
@pytest.mark.parametrize("act, affine", [(None, True), ("silu", True), ("relu", True), ("silu", False)])
def test_layer_norm_backward(n, c, dtype, act, affine):
    g = gen(n * 1000 + c + 1)
    x = normal(g, n, c, dtype=dtype, scale=2.0, shift=1.5)
    gamma = normal(g, c, dtype=dtype, scale=0.3, shift=1.0) if affine else None
    beta = normal(g, c, dtype=dtype, scale=0.3) if affine else None
    dy = normal(g, n, c, dtype=dtype)
    stats = torch.empty(n, 2, device="cuda")
    smc.layer_norm(x, gamma, beta, act=act, stats=stats)
    _, z, xh, mean, rstd, _ = norm_ref(x, gamma, beta, None, act, stats)
    if act == "relu":
        dy = torch.where(z.abs() < 1e-4, 0.0, dy.double()).to(dtype)  # no gradient where the kink's side is a rounding
    dx, dgamma, dbeta = smc.layer_norm_backward(dy, x, stats, gamma, beta, act=act)
    s = torch.sigmoid(z)
    dz = dy.double() * ((z > 0).double() if act == "relu" else s * (1 + z * (1 - s)) if act == "silu" else 1.0)
    gg = dz * gamma.double() if affine else dz
    m1, m2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    ref = rstd * (gg - m1 - xh * m2)
    near = (x.double().abs() + mean.abs()) * rstd + 2  # what an ulp of x does to xh, and to the slope
    mag = dy.double().abs() * 1.1 * (gamma.double().abs() if affine else 1.0)
    err = 64 * E * rstd * (mag + mag.mean(1, keepdim=True) + xh.abs() * (mag * xh.abs()).mean(1, keepdim=True)) * near \
        + 64 * E * rstd * ((mag * near).mean(1, keepdim=True) * (1 + xh.abs()))
    close(dx, ref, u_of(dtype) * ref.abs() + err + 1e-7 * (dtype == F16), "dx")
    if not affine:
        assert dgamma is None and dbeta is None
        return
    for got, terms in ((dgamma, dz * xh), (dbeta, dz)):
        t = terms.sum(0)
        close(got, t, u_of(dtype) * t.abs() + 64 * E * (dy.double().abs() * 1.1 * (near + xh.abs())).sum(0)
              + 1e-7 * (dtype == F16), "sums")


# dbeta of a constant dy whose fp32 running sum would lose nearly half a step with
# each of its later rows: no more than 512 rows in one running sum of fp32, which
# is then off by at most 512 / 2 times 2^-24 of itself (each addition by half a
# step of the sum so far); a block's rows and warps add a few more.
def test_layer_norm_gradient_sums_of_many_rows():
    n, c = 114_000_000, 3  # 4000 rows to a group of lanes of a grid that fits the machine once
    step = 1 + 2.0 ** -13 - 2.0 ** -23
    x = torch.zeros(n, c, device="cuda")
    x[:, 0] = 1.0
    dy = torch.full((n, c), step, device="cuda")
    st = torch.empty(n, 2, device="cuda")
    smc.layer_norm(x, out=torch.empty_like(x), stats=st)
    dbeta, dgamma = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    smc.layer_norm_backward(dy, x, st, dx=dy, dgamma=dgamma, dbeta=dbeta)
    tol = (512 / 2 + 16) * E
    assert float((dbeta.double() / (n * step) - 1).abs().max()) <= tol
    xh = (x[0].double() - st[0, 0].double()) * st[0, 1].double()
    assert float((dgamma.double() / (n * step * xh) - 1).abs().max()) <= tol + 8 * E


def test_layer_norm_gradient_sums_of_many_wide_rows():
    n, c = 400_000, 1030  # 6250 rows to each of 64 slices
    step = 1 + 2.0 ** -12 - 2.0 ** -23
    x = torch.zeros(n, c, device="cuda")
    x[:, ::2] = 1.0
    dy = torch.full((n, c), step, device="cuda")
    st = torch.empty(n, 2, device="cuda")
    smc.layer_norm(x, out=torch.empty_like(x), stats=st)
    dbeta, dgamma = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    smc.layer_norm_backward(dy, x, st, dx=dy, dgamma=dgamma, dbeta=dbeta)
    tol = (512 / 2 + 16) * E
    assert float((dbeta.double() / (n * step) - 1).abs().max()) <= tol
    xh = (x[0].double() - st[0, 0].double()) * st[0, 1].double()
    assert float((dgamma.double() / (n * step * xh) - 1).abs().max()) <= tol + 8 * E


def test_layer_norm_in_place_strided_and_unaligned():
    g = gen(5)
    for dtype in (F32, BF16):
        base = normal(g, 100, 72, dtype=dtype)
        x = base[:, 3:67]  # rows neither dense nor aligned
        ref = smc.layer_norm(x.contiguous())
        assert torch.equal(smc.layer_norm(x), ref)
        flat = normal(g, 100 * 64 + 1, dtype=dtype)
        odd = flat[1:].view(100, 64)  # dense, but off the 16-byte boundary
        ref = smc.layer_norm(odd.clone())
        assert torch.allclose(smc.layer_norm(odd).float(), ref.float(), rtol=2 * u_of(dtype), atol=1e-6)
        y = odd.clone()
        assert smc.layer_norm(y, out=y) is y and torch.equal(y, ref)
        st = torch.empty(100, 2, device="cuda")
        smc.layer_norm(odd.clone(), stats=st)
        dy = normal(g, 100, 64, dtype=dtype)
        dx, _, _ = smc.layer_norm_backward(dy, odd.clone(), st)
        d2 = dy.clone()
        smc.layer_norm_backward(d2, odd.clone(), st, dx=d2)
        assert torch.equal(d2, dx)
        x2 = odd.clone()
        smc.layer_norm_backward(dy, x2, st, dx=x2)
        assert torch.equal(x2, dx)
    with pytest.raises(ValueError):
        smc.layer_norm(base[:, 3:67], out=base[:, 3:67])


def test_layer_norm_rows_do_not_mix():
    g = gen(6)
    x = normal(g, 64, 128, dtype=BF16)
    ref = smc.layer_norm(x)
    x[5, 3], x[9] = math.nan, math.inf
    y = smc.layer_norm(x)
    keep = [i for i in range(64) if i not in (5, 9)]
    assert torch.equal(y[keep], ref[keep]) and bool(y[5].isnan().all()) and bool(y[9].isnan().all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_layer_norm_silu_far_out(dtype):
    """Behind the cut of the exponential: the values and slopes of far negative
    arguments vanish however far they are, and a NaN stays in its channel."""
    g = gen(61)
    big = 3e4 if dtype == F16 else 1e30
    x = normal(g, 37, 64, dtype=dtype)
    gamma = torch.full((64,), big, dtype=dtype, device="cuda")
    gamma[10], gamma[30] = math.nan, 1.0
    stats = torch.empty(37, 2, device="cuda")
    y = smc.layer_norm(x, gamma, act="silu", stats=stats)
    assert bool(y[:, 10].isnan().all()) and not bool(y[:, 9].isnan().any()) and not bool(y[:, 11].isnan().any())
    z = gamma.double() * (x.double() - stats[:, :1]) * stats[:, 1:]
    far = z < -100
    assert int(far.sum()) > 500 and float(y[far].double().abs().max()) < 1e-16
    gamma[10] = big
    far[:, 10] = False
    near = torch.zeros_like(far)
    near[:, 30] = True
    dy = torch.where(far | near, normal(g, 37, 64, dtype=dtype), 0.0).to(dtype)
    only = torch.where(near, dy, 0.0).to(dtype)
    a = smc.layer_norm_backward(dy, x, stats, gamma, act="silu")
    b = smc.layer_norm_backward(only, x, stats, gamma, act="silu")
    # what the slopes behind the cut (below 1e-17, times gamma) add to dx and dgamma
    assert float((a[0].double() - b[0].double()).abs().max()) <= 1e-15 * big
    assert float((a[1].double() - b[1].double()).abs().max()) <= 1e-15


def test_layer_norm_no_rows():
    x = torch.empty(0, 16, device="cuda")
    assert smc.layer_norm(x).shape == (0, 16)
    w = torch.ones(16, device="cuda")
    dx, dg, db = smc.layer_norm_backward(x, x, torch.empty(0, 2, device="cuda"), w, w)
    assert dx.shape == (0, 16) and not dg.any() and not db.any()


def test_layer_norm_gradient_against_differences():
    g = gen(7)
    x, dy = normal(g, 5, 24), normal(g, 5, 24)
    gamma, beta = normal(g, 24, scale=0.2, shift=1.0), normal(g, 24, scale=0.2)
    st = torch.empty(5, 2, device="cuda")
    smc.layer_norm(x, gamma, beta, act="silu", stats=st)
    grads = smc.layer_norm_backward(dy, x, st, gamma, beta, act="silu")

    def loss(x, gamma, beta):
        return float((norm_ref(x, gamma, beta, 1e-5, "silu")[0] * dy.double()).sum())

    args = [t.double() for t in (x, gamma, beta)]
    h = 1e-5
    for k, got in enumerate(grads):
        for i in torch.randperm(args[k].numel(), generator=torch.Generator().manual_seed(k))[:12].tolist():
            up, down = [t.clone() for t in args], [t.clone() for t in args]
            up[k].view(-1)[i] += h
            down[k].view(-1)[i] -= h
            d = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(float(got.reshape(-1)[i]) - d) <= 1e-5 * (1 + abs(d)), (k, i)


# ---------------------------------------------------------------------- rotary
def rotary_ref(x, pos, freqs, layout, scale, inverse):
    ang = (pos.double()[:, :, None] * freqs).flatten(1)[:, None]
    c, s = torch.cos(ang) * scale, torch.sin(ang) * (-scale if inverse else scale)
    x = x.double()
    p = ang.shape[-1]
    y, tol = x.clone(), torch.zeros_like(x)
    u, v = (x[..., :p], x[..., p:2 * p]) if layout == "half" else (x[..., 0:2 * p:2], x[..., 1:2 * p:2])
    t = 8 * E * abs(scale) * (u.abs() + v.abs())  # angle, sine and cosine: under 2^-22 each; two products
    iu, iv = (slice(0, p), slice(p, 2 * p)) if layout == "half" else (slice(0, 2 * p, 2), slice(1, 2 * p, 2))
    y[..., iu], y[..., iv] = u * c - v * s, u * s + v * c
    tol[..., iu], tol[..., iv] = t, t
    return y, tol


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n, h, d, axes, pairs, far", [
    (1, 1, 2, 1, 1, 10), (3, 8, 128, 1, 32, 2 ** 31 - 1), (1000, 4, 64, 3, 10, 64), (77, 3, 64, 1, 32, 4096),
    (5, 2, 40, 2, 7, 1000000), (13, 5, 33, 1, 16, 100), (9, 1, 96, 3, 16, 512), (2, 70, 24, 2, 4, 50),
    (30000, 2, 16, 1, 8, 1000)])
def test_rotary(n, h, d, axes, pairs, far, layout, dtype):
    g = gen(n + d)
    x = normal(g, n, h, d, dtype=dtype)
    coords = torch.randint(-far, far, (n, 1 + axes), generator=g, device="cuda").to(torch.int32)
    pos = coords[:, 1:]
    freqs, _ = smc.rotary_freqs(pairs, axes, device="cuda")
    for scale, inverse in ((1.0, False), (1.2, True)):
        y = smc.rotary(x, pos, freqs, layout=layout, scale=scale, inverse=inverse)
        ref, tol = rotary_ref(x, pos, freqs, layout, scale, inverse)
        close(y, ref, u_of(dtype) * ref.abs() * (tol > 0) + tol + 6e-8 * (dtype == F16), "rotary")
        if 2 * axes * pairs < d:
            assert torch.equal(y[..., 2 * axes * pairs:], x[..., 2 * axes * pairs:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_views(layout):
    g = gen(11)
    qkv = normal(g, 50, 3, 4, 32, dtype=BF16)
    pos = torch.randint(0, 100, (50, 4), generator=g, device="cuda").to(torch.int32)[:, 1:]
    freqs, _ = smc.rotary_freqs(4, 3, device="cuda")
    kw = dict(positions=pos, freqs=freqs, layout=layout)
    ref = smc.rotary(qkv[:, 1].contiguous(), **kw)
    assert torch.equal(smc.rotary(qkv[:, 1], **kw), ref)
    assert torch.equal(smc.rotary(qkv[:, 1], positions=pos.contiguous(), freqs=freqs, layout=layout), ref)
    t = qkv[:, 1].transpose(1, 2).contiguous().transpose(1, 2)  # the last axis not dense
    assert torch.equal(smc.rotary(t, **kw), ref)
    hm = qkv[:, 1].transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    assert torch.equal(smc.rotary(hm, **kw), ref)
    odd = normal(g, 50, 4, 33, dtype=BF16)[..., :32]  # rows off the 16-byte boundary
    assert torch.equal(smc.rotary(odd, **kw), smc.rotary(odd.contiguous(), **kw))
    same = qkv[:1, 1].expand(50, 4, 32)  # a broadcast input
    assert torch.equal(smc.rotary(same, **kw), smc.rotary(same.contiguous(), **kw))
    packed = qkv.clone()
    smc.rotary(packed[:, 1], out=packed[:, 1], **kw)  # in place, in the packed buffer
    assert torch.equal(packed[:, 1], ref) and torch.equal(packed[:, 0], qkv[:, 0]) and torch.equal(packed[:, 2], qkv[:, 2])
    with pytest.raises(smc.SmcError) as e:
        smc.rotary(packed[:, 1], out=packed[:, 1, :1].expand(50, 4, 32), **kw)
    assert e.value.name == "SMC_E_ARG"
    with pytest.raises(smc.SmcError) as e:
        smc.rotary(packed.view(50, 12, 32)[:, 0:4], out=packed.view(50, 12, 32)[:, 1:5], **kw)
    assert e.value.name == "SMC_E_ALIAS"
    assert smc.rotary(qkv[:0, 1], positions=pos[:0], freqs=freqs, layout=layout).shape == (0, 4, 32)


# ------------------------------------------------------------------- attention
def spans(offsets):
    o = offsets.tolist()
    return list(zip(o[:-1], o[1:]))


def attention_ref(q, k, v, qo, ko, scale, causal, dout=None, out=None, lse=None):
    """Outputs and tolerances in 64 bits, item by item and head by head."""
    t = q.dtype
    u = u_of(t)
    pu = 0.0 if t == F32 else u  # P and dS are rounded to the inputs' type
    n, h, d = q.shape
    hk = k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    r = {x: torch.zeros(n, h, d, dtype=torch.float64, device="cuda") for x in ("out", "dq", "tout", "tdq")}
    r |= {x: torch.zeros(k.shape[0], hk, d, dtype=torch.float64, device="cuda") for x in ("dk", "dv", "tdk", "tdv")}
    r["lse"] = torch.full((n, h), -math.inf, dtype=torch.float64, device="cuda")
    r["tlse"] = torch.zeros_like(r["lse"])
    for (a, b), (c, e) in zip(spans(qo), spans(ko)):
        if a == b or c == e:
            continue
        for i in range(h):
            j = i // (h // hk)
            Q, K, V = q[a:b, i], k[c:e, j], v[c:e, j]
            s = scale * Q @ K.T
            # products and sums of d terms in fp32, the scale, the subtraction and the exponential
            se = E * ((d / 4 + 8) * scale * Q.abs() @ K.abs().T + 8 * s.abs() + 16)
            if causal:
                hide = torch.ones_like(s, dtype=torch.bool).triu((e - c) - (b - a) + 1)
                s = s.masked_fill(hide, -math.inf)
                se = se.masked_fill(hide, 0.0)
            if dout is None:
                seen = (s > -math.inf).any(1, keepdim=True)
                l = torch.logsumexp(s, 1, keepdim=True)
                p = torch.exp(s - l.masked_fill(~seen, 0.0))
                r["out"][a:b, i] = p @ V
                worst = se.amax(1, keepdim=True)
                pe = 4 * worst + 4 * E * l.masked_fill(~seen, 0.0).abs() + 2 * E * math.sqrt(e - c)
                r["tout"][a:b, i] = u * r["out"][a:b, i].abs() + (pu + pe) * (p @ V.abs())
                r["lse"][a:b, i] = l[:, 0]
                r["tlse"][a:b, i] = (2 * worst + 8 * E * (1 + l.masked_fill(~seen, 0.0).abs()))[:, 0]
                continue
            l = lse[a:b, i].double()[:, None]
            p = torch.exp(s - l.masked_fill(l == -math.inf, 0.0))
            pe = se + 4 * E * l.masked_fill(l == -math.inf, 0.0).abs()
            dO, O = dout[a:b, i].double(), out[a:b, i].double()
            dp = dO @ V.T
            delta = (dO * O).sum(1, keepdim=True)
            ds = p * (dp - delta)
            de = E * (d / 4 + 8) * (dO.abs() @ V.abs().T + (dO.abs() * O.abs()).sum(1, keepdim=True))
            dse = (pu + 2 * pe) * ds.abs() + p * de
            if t == F16:  # the scaled dS keeps at least 2^-24 of its bound
                dse = dse + 2.0 ** -36 * float((dO.norm(dim=1).max() * V.norm(dim=1).max()))
            r["dq"][a:b, i] = scale * ds @ K
            r["tdq"][a:b, i] = scale * dse @ K.abs()
            r["dk"][c:e, j] += scale * ds.T @ Q
            r["tdk"][c:e, j] += scale * dse.T @ Q.abs()
            r["dv"][c:e, j] += p.T @ dO
            r["tdv"][c:e, j] += ((pu + 2 * pe) * p).T @ dO.abs()
    acc = 2 * E * 8  # sums over rows and keys, held in fp32
    for x in ("dq", "dk", "dv"):
        r["t" + x] = r["t" + x] * (1 + acc) + u * r[x].abs()
        r["t" + x] += 32 * E * r["t" + x].clamp_min(0).mean() + 16 * E * r[x].abs()
    floor = 6e-8 if t == F16 else 0.0
    for x in ("out", "dq", "dk", "dv"):
        r["t" + x] += floor + 1e-30
    return r


def offsets_of(rows, first=0):
    return torch.tensor([first] + [first + sum(rows[:i + 1]) for i in range(len(rows))], dtype=torch.int32, device="cuda")


# queries, keys of each item (None: the queries'), heads, kv heads, dim, causal
ATTENTION = [
    ([1], None, 1, 1, 8, False), ([1], [1], 2, 1, 64, True), ([5, 0, 3], [0, 4, 7], 2, 2, 64, False),
    ([127, 1, 128], None, 2, 2, 64, False), ([129], [63], 4, 2, 64, True), ([64, 200], [65, 300], 3, 1, 64, True),
    ([256, 257, 255], None, 2, 1, 128, True), ([300], [700], 6, 2, 128, False), ([1, 1, 1], [1000, 1, 33], 8, 2, 128, False),
    ([3, 2], [900, 5], 8, 1, 64, True), ([513], None, 1, 1, 40, False), ([70, 33], [70, 0], 2, 2, 24, False),
    ([90], [130], 2, 2, 7, False), ([65], None, 2, 1, 1, True), ([1200], None, 2, 2, 96, True), ([130], [257], 5, 5, 80, False),
    ([9, 40], [50, 60], 64, 1, 16, True), ([33], [65], 7, 1, 32, True), ([200], [100], 3, 3, 120, True),
    ([2100], [1900], 1, 1, 64, False), ([17] * 40, None, 2, 2, 64, False), ([1, 2, 3, 4, 5] * 70, [5, 4, 3, 2, 1] * 70, 4, 2, 32, True),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention_and_gradients(case, dtype):
    ql, kl, h, hk, d, causal = ATTENTION[case]
    g = gen(case)
    qo = offsets_of(ql)
    ko = None if kl is None else offsets_of(kl)
    q = normal(g, sum(ql), h, d, dtype=dtype)
    k, v = (normal(g, sum(kl or ql), hk, d, dtype=dtype) for _ in range(2))
    dout = normal(g, sum(ql), h, d, dtype=dtype)
    lse = torch.full((sum(ql), h), math.nan, device="cuda")
    out = smc.attention(q, k, v, qo, ko, causal=causal, lse=lse)
    ko_ = qo if ko is None else ko
    r = attention_ref(q, k, v, qo, ko_, d ** -0.5, causal)
    close(out, r["out"], r["tout"], "out")
    empty = r["lse"] == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    close(torch.where(empty, 0.0, lse), torch.where(empty, 0.0, r["lse"]), r["tlse"], "lse")
    assert torch.equal(smc.attention(q, k, v, qo, ko, causal=causal), out)  # without lse: the same bits
    got = smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal)
    b = attention_ref(q, k, v, qo, ko_, d ** -0.5, causal, dout, out, lse)
    for x, y in zip(("dq", "dk", "dv"), got):
        close(y, b[x], b["t" + x], x)
    again = smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal)
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    smc.status()


# many short items: a block then works through several heads; long rows of few
# items: keys (forward) and queries (gradients) are split between blocks
MANY = [([i * 7 % 23 for i in range(1300)], None, 5, 5, 64, False), ([i * 11 % 190 for i in range(400)], None, 20, 20, 128, False),
        ([i * 5 % 140 for i in range(700)], [i * 13 % 90 for i in range(700)], 16, 8, 40, True),
        ([700], [6000], 4, 2, 64, False), ([5000, 3, 0, 64], None, 4, 1, 128, True), ([3000], [400], 2, 2, 64, True),
        ([400], [3000], 2, 1, 72, True), ([6000, 10], [130, 0], 8, 1, 64, False)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_many_items_and_splits(case, dtype):
    ql, kl, h, hk, d, causal = MANY[case]
    g = gen(100 + case)
    qo, ko = offsets_of(ql), offsets_of(kl or ql)
    q, dout = (normal(g, sum(ql), h, d, dtype=dtype) for _ in range(2))
    k, v = (normal(g, sum(kl or ql), hk, d, dtype=dtype) for _ in range(2))
    lse = torch.empty(sum(ql), h, device="cuda")
    out = smc.attention(q, k, v, qo, ko, causal=causal, lse=lse)
    got = smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal)
    smc.status()
    few = len(ql) > 100  # the plain form goes item by item: take every 37th of many
    for i in range(0, len(ql), 37 if few else 1):
        (a, b), (c, e) = spans(qo[i:i + 2])[0], spans(ko[i:i + 2])[0]
        if a == b or c == e:
            assert not out[a:b].any() and bool((lse[a:b] == -math.inf).all())
            assert not got[0][a:b].any() and not got[1][c:e].any() and not got[2][c:e].any()
            continue
        one = (q[a:b], k[c:e], v[c:e], offsets_of([b - a]), offsets_of([e - c]), d ** -0.5, causal)
        r = attention_ref(*one)
        close(out[a:b], r["out"], r["tout"], "out")
        r = attention_ref(*one, dout[a:b], out[a:b], lse[a:b])
        for x, y in zip(("dq", "dk", "dv"), (got[0][a:b], got[1][c:e], got[2][c:e])):
            close(y, r[x], r["t" + x], x)
    assert torch.equal(out, smc.attention(q, k, v, qo, ko, causal=causal))
    again = smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_tens_of_thousands_of_items(dtype):
    """More items than a block looks at in several rounds (768 to 2304 of them a
    round), empty ones among them; sampled against the plain form."""
    rows = [i * 7 % 6 for i in range(30_011)]
    g = gen(430)
    o = torch.tensor([0] + rows).cumsum(0).to(torch.int32).cuda()
    n = sum(rows)
    q, k, v, dout = (normal(g, n, 2, 64, dtype=dtype) for _ in range(4))
    lse = torch.empty(n, 2, device="cuda")
    out = smc.attention(q, k, v, o, lse=lse)
    got = smc.attention_backward(dout, q, k, v, out, lse, o)
    smc.status()
    ends = o.tolist()
    for i in [0, 1, 766, 767, 768, 769, 1535, 1536, 2303, 2304, 2305, 6912, 9999, 20_000, 29_999, 30_009, 30_010]:
        a, b = ends[i], ends[i + 1]
        if a == b:
            continue
        one = offsets_of([b - a])
        r = attention_ref(q[a:b], k[a:b], v[a:b], one, one, 64 ** -0.5, False)
        close(out[a:b], r["out"], r["tout"], "out")
        r = attention_ref(q[a:b], k[a:b], v[a:b], one, one, 64 ** -0.5, False, dout[a:b], out[a:b], lse[a:b])
        for x, y in zip(("dq", "dk", "dv"), got):
            close(y[a:b], r[x], r["t" + x], x)


# splits of the FMA kernels: groups that do not divide a tile, odd widths, items
# of different lengths, keys that no query sees
@pytest.mark.parametrize("ql, kl, h, hk, d, causal, dtype", [
    ([1000, 7], [300, 900], 3, 1, 33, False, F32), ([1000, 7], [300, 900], 3, 1, 33, True, BF16),
    ([500], [2000], 5, 1, 20, True, F16), ([2000, 0, 90], [500, 30, 0], 7, 1, 128, True, F32),
    ([63], [129], 1, 1, 96, False, F32), ([1], [4000], 2, 2, 64, False, F32), ([4000], [1], 2, 2, 16, True, F32)])
def test_attention_gradients_of_split_rows(ql, kl, h, hk, d, causal, dtype):
    g = gen(300 + d)
    qo, ko = offsets_of(ql), offsets_of(kl)
    q, dout = (normal(g, sum(ql), h, d, dtype=dtype) for _ in range(2))
    k, v = (normal(g, sum(kl), hk, d, dtype=dtype) for _ in range(2))
    lse = torch.empty(sum(ql), h, device="cuda")
    out = smc.attention(q, k, v, qo, ko, causal=causal, lse=lse)
    got = smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal)
    r = attention_ref(q, k, v, qo, ko, d ** -0.5, causal, dout, out, lse)
    for x, y in zip(("dq", "dk", "dv"), got):
        close(y, r[x], r["t" + x], x)
    again = smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal)
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    smc.status()


def test_attention_gradients_of_long_sums():
    """12,000 packed rows in one fp32 sum: 188 sums of 64.  Each term is off by
    about 8 x 2^-24 (its score's and its exponent's rounding), independently of
    the others; the roundings of the sums of 64 and of their sum add, as a random
    walk over growing partial sums, at most sqrt(64) and sqrt(188) times 2^-24 of
    them: sqrt(8^2 + 8^2 + 14^2) = 18 x 2^-24 in the norm."""
    g = gen(330)
    o = offsets_of([3000])
    q, dout = normal(g, 3000, 4, 64), normal(g, 3000, 4, 64)
    k, v = normal(g, 3000, 1, 64), normal(g, 3000, 1, 64)
    lse = torch.empty(3000, 4, device="cuda")
    out = smc.attention(q, k, v, o, causal=True, lse=lse)
    got = smc.attention_backward(dout, q, k, v, out, lse, o, causal=True)
    r = attention_ref(q, k, v, o, o, 64 ** -0.5, True, dout, out, lse)
    for x, y in zip(("dq", "dk", "dv"), got):
        assert float((y.double() - r[x]).norm() / r[x].norm()) <= 18 * E, x


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 20])
def test_attention_rows_outside_items(dtype, d):
    """Rows before, between and behind the items hold NaN and infinities: they
    reach no output, and their own outputs are left as they were."""
    g = gen(d)
    ql, kl, h, hk = [100, 0, 37], [61, 5, 200], 4, 2
    qo, ko = offsets_of(ql, 9), offsets_of(kl, 3)
    n, m = 9 + sum(ql) + 150, 3 + sum(kl) + 140
    q, k, v, dout = (normal(g, a, b, d, dtype=dtype) for a, b in ((n, h), (m, hk), (m, hk), (n, h)))
    for t, lo, hi in ((q, 9, 146), (k, 3, 269), (v, 3, 269), (dout, 9, 146)):
        t[:lo] = math.nan
        t[hi:] = math.inf
    out, lse = torch.full_like(q, 7.0), torch.full((n, h), 7.0, device="cuda")
    assert smc.attention(q, k, v, qo, ko, out=out, lse=lse) is out
    r = attention_ref(q[9:146], k[3:269], v[3:269], qo - 9, ko - 3, d ** -0.5, False)
    close(out[9:146], r["out"], r["tout"], "out")
    for t in (out, lse):
        assert bool((t[:9] == 7).all()) and bool((t[146:] == 7).all())
    grads = [torch.full_like(t, 5.0) for t in (q, k, v)]
    smc.attention_backward(dout, q, k, v, out, lse, qo, ko, dq=grads[0], dk=grads[1], dv=grads[2])
    b = attention_ref(q[9:146], k[3:269], v[3:269], qo - 9, ko - 3, d ** -0.5, False, dout[9:146], out[9:146], lse[9:146])
    for x, t, lo, hi in (("dq", grads[0], 9, 146), ("dk", grads[1], 3, 269), ("dv", grads[2], 3, 269)):
        close(t[lo:hi], b[x], b["t" + x], x)
        assert bool((t[:lo] == 5).all()) and bool((t[hi:] == 5).all())
    assert not grads[1][64:69].any() and not grads[2][64:69].any()  # keys that no query has


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_views(dtype, d):
    g = gen(20 + d)
    n, h = 150, 2
    qkv = normal(g, n, 3, h, d, dtype=dtype)
    o = offsets_of([70, 80])
    q, k, v = qkv.unbind(1)
    dense = [t.contiguous() for t in (q, k, v)]
    lse = torch.empty(n, h, device="cuda")
    out = smc.attention(*dense, o, lse=lse)
    assert torch.equal(smc.attention(q, k, v, o), out)
    heads_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in dense]
    assert torch.equal(smc.attention(*heads_first, o), out)
    odd = [torch.nn.functional.pad(t, (1, 0))[..., 1:] for t in dense]  # off the 16-byte boundary
    r = attention_ref(*dense, o, o, d ** -0.5, False)
    close(smc.attention(*odd, o), r["out"], r["tout"], "unaligned")
    dout = normal(g, n, h, d, dtype=dtype)
    ref = smc.attention_backward(dout, *dense, out, lse, o)
    packed = torch.full_like(qkv, 3.0)
    smc.attention_backward(dout, q, k, v, out, lse, o, dq=packed[:, 0], dk=packed[:, 1], dv=packed[:, 2])
    assert all(torch.equal(packed[:, i], ref[i]) for i in range(3))
    got = smc.attention_backward(dout[:1].expand(n, h, d), q, k, v, out, lse, o)
    want = smc.attention_backward(dout[:1].expand(n, h, d).contiguous(), q, k, v, out, lse, o)
    b = attention_ref(*dense, o, o, d ** -0.5, False, dout[:1].expand(n, h, d), out, lse)
    for x, y, z in zip(("dq", "dk", "dv"), got, want):
        close(y, b[x], b["t" + x], x)
        close(z, b[x], b["t" + x], x)
    one = k[:, :1].expand(n, h, d)  # one head broadcast to all
    close(smc.attention(q, one, one, o), *(lambda a: (a["out"], a["tout"]))(attention_ref(q, one, one, o, o, d ** -0.5, False)), "bc")
    with pytest.raises(smc.SmcError) as e:
        smc.attention(q, k, v, o, out=qkv.view(-1)[:n * h * d].view(n, h, d))
    assert e.value.name == "SMC_E_ALIAS"


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_bad_offsets_are_cut_and_reported(dtype):
    g = gen(30)
    q = normal(g, 200, 2, 64, dtype=dtype)
    lse = torch.empty(200, 2, device="cuda")
    smc.status()
    for bad in ([0, 300], [-5, 100], [0, 150, 100, 200], [400, 500], [0, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1]):
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out = smc.attention(q, q, q, o, lse=lse)
        with pytest.raises(smc.SmcError) as e:
            smc.status()
        assert e.value.name == "SMC_E_RANGE", bad
        smc.attention_backward(q, q, q, q, out, lse, o)
        with pytest.raises(smc.SmcError):
            smc.status()
    smc.attention(q, q, q, offsets_of([200]))
    smc.status()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n, m, causal", [(0, 1500, False), (1500, 0, True), (0, 5, True), (3, 0, False)])
def test_attention_with_one_side_empty(n, m, causal, dtype):
    """No queries, or no keys, in the whole call: gradients of what is there are zero."""
    g = gen(450)
    qo, ko = offsets_of([n]), offsets_of([m])
    q, dout = normal(g, n, 4, 64, dtype=dtype), normal(g, n, 4, 64, dtype=dtype)
    k, v = normal(g, m, 2, 64, dtype=dtype), normal(g, m, 2, 64, dtype=dtype)
    lse = torch.full((n, 4), math.nan, device="cuda")
    out = smc.attention(q, k, v, qo, ko, causal=causal, lse=lse, out=torch.full_like(q, math.nan))
    assert not out.any() and bool((lse == -math.inf).all())
    grads = [torch.full_like(x, math.nan) for x in (q, k, v)]
    smc.attention_backward(dout, q, k, v, out, lse, qo, ko, causal=causal, dq=grads[0], dk=grads[1], dv=grads[2])
    smc.status()
    assert all(not x.any() for x in grads)


def test_attention_far_rows():
    """Element offsets past 32 bits: rows 2^24 elements apart."""
    g = gen(31)
    n, d, row = 300, 64, 1 << 24
    buf = torch.empty(n * row, dtype=BF16, device="cuda")
    q, k, v = (buf.as_strided((n, 1, d), (row, d, 1), i * 256) for i in range(3))
    for t in (q, k, v):
        t.copy_(normal(g, n, 1, d, dtype=BF16))
    o = offsets_of([n])
    out = smc.attention(q, k, v, o)
    assert torch.equal(out, smc.attention(q.contiguous(), k.contiguous(), v.contiguous(), o))
    turned = torch.empty(n * row, dtype=BF16, device="cuda").as_strided((n, 1, d), (row, d, 1), 1024)
    freqs, _ = smc.rotary_freqs(32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    smc.rotary(q, pos, freqs, out=turned)
    assert torch.equal(turned, smc.rotary(q.contiguous(), pos, freqs))


def test_layer_norm_far_rows():
    g = gen(32)
    n, c = 33_600_000, 64  # 2.15e9 elements
    x = torch.empty(n, c, dtype=BF16, device="cuda")
    tail = normal(g, 1000, c, dtype=BF16)
    x[-1000:] = tail
    x[:-1000] = tail[:1]
    y = smc.layer_norm(x)
    assert torch.equal(y[-1000:], smc.layer_norm(tail))


# fp16 gradients of parts of a call whose dout differ by up to 10^6: per item, per
# key/value head, per query
def _scaled_case(h, hk, d, rows, causal, seed):
    g = gen(seed)
    o = offsets_of(rows)
    n = sum(rows)
    q, dout = normal(g, n, h, d, dtype=F16), normal(g, n, h, d)
    k, v = normal(g, n, hk, d, dtype=F16), normal(g, n, hk, d, dtype=F16)
    lse = torch.empty(n, h, device="cuda")
    return q, k, v, dout, smc.attention(q, k, v, o, causal=causal, lse=lse), lse, o


def _within(got, ref, what):
    """One rounding of dS or P to fp16 under each sum and one of the result: 2 u
    in the norm (the roundings of a sum's terms are independent of each other), and
    half of fp16's smallest step for each element."""
    fits = ref.abs() < 65_000.0  # what leaves fp16's range is infinite
    got, ref = got.double()[fits], ref[fits]
    err, size = float((got - ref).norm()), float(ref.norm())
    assert err <= 2 * u_of(F16) * size + 2.0 ** -25 * math.sqrt(ref.numel()), (what, err / size)


@pytest.mark.parametrize("h, hk, d, rows, causal", [
    (2, 2, 64, [1000, 900], False), (4, 1, 128, [700, 600], True), (2, 2, 64, [40, 30], False),
    (8, 2, 128, [3000, 1000], False), (3, 1, 40, [500, 400], True)])
@pytest.mark.parametrize("small", [1e4, 1.0, 1e-2])
def test_fp16_gradients_of_items_on_their_own_scale(h, hk, d, rows, causal, small):
    q, k, v, dout, out, lse, o = _scaled_case(h, hk, d, rows, causal, 400 + d)
    a = rows[0]
    dout[:a] *= 1e4
    dout[a:] *= small
    dout = dout.clamp(-6e4, 6e4).to(F16)
    got = smc.attention_backward(dout, q, k, v, out, lse, o, causal=causal)
    r = attention_ref(q, k, v, o, o, d ** -0.5, causal, dout, out, lse)
    for x, y in zip(("dq", "dk", "dv"), got):
        _within(y[:a], r[x][:a], x + " of the first item")
        _within(y[a:], r[x][a:], x + " of the second item")


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_gradients_of_heads_and_queries_on_their_own_scale(d):
    q, k, v, dout, out, lse, o = _scaled_case(4, 2, d, [1000], False, 410 + d)
    by_head = dout * torch.tensor([1e4, 1e4, 1e-2, 1e-2], device="cuda")[:, None]
    by_head = by_head.clamp(-6e4, 6e4).to(F16)
    got = smc.attention_backward(by_head, q, k, v, out, lse, o)
    r = attention_ref(q, k, v, o, o, d ** -0.5, False, by_head, out, lse)
    for x, y in zip(("dq", "dk", "dv"), got):
        per = y.shape[1] // 2
        _within(y[:, :per], r[x][:, :per], x + " of the first head")
        _within(y[:, per:], r[x][:, per:], x + " of the second head")
    # by query: dq is each query's own (dk and dv are sums over the queries)
    by_row = dout.clone()
    by_row[::2] *= 1e4
    by_row[1::2] *= 1e-2
    by_row = by_row.clamp(-6e4, 6e4).to(F16)
    got = smc.attention_backward(by_row, q, k, v, out, lse, o)
    r = attention_ref(q, k, v, o, o, d ** -0.5, False, by_row, out, lse)
    _within(got[0][::2], r["dq"][::2], "dq of large rows")
    _within(got[0][1::2], r["dq"][1::2], "dq of small rows")
    _within(got[1], r["dk"], "dk")
    _within(got[2], r["dv"], "dv")


def test_fp16_gradients_with_a_value_row_far_larger():
    """|V| of one item does not reach the other's scale either."""
    q, k, v, dout, _, _, o = _scaled_case(2, 2, 64, [600, 500], False, 420)
    v[:600] *= 5e3
    v[600:] *= 1e-2
    dout = dout.to(F16)
    lse = torch.empty(1100, 2, device="cuda")
    out = smc.attention(q, k, v, o, lse=lse)
    got = smc.attention_backward(dout, q, k, v, out, lse, o)
    r = attention_ref(q, k, v, o, o, 64 ** -0.5, False, dout, out, lse)
    for x, y in zip(("dq", "dk", "dv"), got):
        _within(y[:600], r[x][:600], x + " of the first item")
        _within(y[600:], r[x][600:], x + " of the second item")


# One key far above tens of thousands of equal ones, whose probabilities lie at the
# low end of fp16: P carries 2^7, so each is off by at most half of 2^-24 of 2^-7
# of the row's largest, 2^-32, and the sum over the keys by that many times as much.
@pytest.mark.parametrize("at", [0, 20_000, 39_999])
@pytest.mark.parametrize("above", [17.5, 17.25, 12.0])
@pytest.mark.parametrize("queries, h, hk, d", [(1, 4, 1, 128), (300, 2, 2, 64), (1300, 2, 1, 128), (2500, 1, 1, 64)])
def test_fp16_attention_keeps_small_probabilities(queries, h, hk, d, above, at):
    keys = 40_000
    q = torch.zeros(queries, h, d, dtype=F16, device="cuda")
    q[..., 0] = 4.0
    k, v = torch.zeros(keys, hk, d, dtype=F16, device="cuda"), torch.ones(keys, hk, d, dtype=F16, device="cuda")
    k[at, :, 0], v[at] = above / 4, 0.0  # exact in fp16
    lse = torch.empty(queries, h, device="cuda")
    out = smc.attention(q, k, v, offsets_of([queries]), offsets_of([keys]), scale=1.0, lse=lse)
    low = (keys - 1) * math.exp(-above)
    ref = low / (1 + low)
    assert float((out.double() - ref).abs().max()) <= (u_of(F16) + 256 * E) * ref + keys * 2.0 ** -32
    assert float((lse.double() - (above + math.log1p(low))).abs().max()) <= 64 * E * above


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["packed rows", "heads in turn", "packed heads"])
def test_attention_gradients_into_one_buffer(layout, dtype):
    g = gen(440)
    n, h, d = 500, 3, 64
    q, k, v, dout = (normal(g, n, h, d, dtype=dtype) for _ in range(4))
    o = offsets_of([300, 200])
    lse = torch.empty(n, h, device="cuda")
    out = smc.attention(q, k, v, o, lse=lse)
    ref = smc.attention_backward(dout, q, k, v, out, lse, o)
    if layout == "packed rows":
        views = torch.empty(n, 3 * h, d, dtype=dtype, device="cuda").split(h, 1)
    elif layout == "heads in turn":
        views = torch.empty(n, h, 3, d, dtype=dtype, device="cuda").unbind(2)
    else:
        views = [t.transpose(0, 1) for t in torch.empty(h, 3, n, d, dtype=dtype, device="cuda").unbind(1)]
    got = smc.attention_backward(dout, q, k, v, out, lse, o, dq=views[0], dk=views[1], dv=views[2])
    assert all(torch.equal(a, b) and a.data_ptr() == c.data_ptr() for a, b, c in zip(got, ref, views))


# ------------------------------------------------ streams, graphs, failures
def _chain(q, k, v, dout, o, pos, freqs, gamma, beta, stream=None):
    n, h, d = q.shape
    st, lse = torch.empty(n, 2, device="cuda"), torch.empty(n, h, device="cuda")
    x = smc.layer_norm(q.view(n, h * d), gamma, beta, act="silu", stats=st, stream=stream)
    qr = smc.rotary(x.view(n, h, d), pos, freqs, stream=stream)
    out = smc.attention(qr, k, v, o, lse=lse, stream=stream)
    dq, dk, dv = smc.attention_backward(dout, qr, k, v, out, lse, o, stream=stream)
    dx = smc.rotary(dq, pos, freqs, inverse=True, stream=stream)
    grads = smc.layer_norm_backward(dx.view(n, h * d), q.view(n, h * d), st, gamma, beta, act="silu", stream=stream)
    return [out, dk, dv, *grads]


def _chain_inputs(seed, dtype=BF16):
    g = gen(seed)
    n, h, d = 500, 2, 64
    q, k, v, dout = (normal(g, n, h, d, dtype=dtype) for _ in range(4))
    pos = torch.randint(0, 64, (n, 3), generator=g, device="cuda").to(torch.int32)
    freqs, _ = smc.rotary_freqs(10, 3, device="cuda")
    return q, k, v, dout, offsets_of([200, 300]), pos, freqs, normal(g, h * d, dtype=dtype), normal(g, h * d, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_streams_and_graphs(dtype):
    a, b = _chain_inputs(1, dtype), _chain_inputs(2, dtype)
    ra, rb = _chain(*a), _chain(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):  # two calls at once, by stream argument and by current stream
        ga = _chain(*a, stream=s1)
        with torch.cuda.stream(s2):
            gb = _chain(*b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ga + gb, ra + rb))
    graphs, outs = [], []
    for inputs in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_chain(*inputs))
        graphs.append(gr)
    for _ in range(3):  # replayed beside each other: they share no scratch
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs[0] + outs[1], ra + rb))
    smc.status()


FIRST_CALL = """
import torch
import submanifold_sparse_convolution_packed_b200 as smc
g = torch.Generator(device="cuda").manual_seed(1)
q, k, v, d = (torch.randn(300, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(4))
x, w = q.view(300, 128), torch.ones(128, dtype=torch.bfloat16, device="cuda")
o = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
st, lse = torch.empty(300, 2, device="cuda"), torch.empty(300, 2, device="cuda")
torch.cuda.synchronize()

def calls():
    out = smc.attention(q, k, v, o, lse=lse)
    y = smc.layer_norm(x, w, w, stats=st)
    return [out, y, *smc.attention_backward(d, q, k, v, out, lse, o), *smc.layer_norm_backward(x, x, st, w, w)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
smc.status()
print("ok")
"""


def test_first_call_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_two_threads_at_once():
    sets = [_chain_inputs(s) for s in (20, 21)]
    refs = [_chain(*i) for i in sets]
    torch.cuda.synchronize()
    outs, errors = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    outs[i] = _chain(*sets[i])
            s.synchronize()
        except Exception as e:  # the main thread reports it
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for got, ref in zip(outs, refs):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    smc.status()


def test_allocation_failures():
    q, k, v, dout, o, *_ = _chain_inputs(3)
    lse = torch.empty(500, 2, device="cuda")
    out = smc.attention(q, k, v, o, lse=lse)
    ref = smc.attention_backward(dout, q, k, v, out, lse, o)
    smc.set_alloc_fail_after(1)
    with pytest.raises(smc.SmcError) as e:
        smc.attention_backward(dout, q, k, v, out, lse, o)
    assert e.value.name == "SMC_E_OOM"
    x, st = q.view(500, 128), torch.empty(500, 2, device="cuda")
    w = torch.ones(128, dtype=BF16, device="cuda")
    smc.layer_norm(x, stats=st)
    smc.set_alloc_fail_after(1)
    with pytest.raises(smc.SmcError) as e:
        smc.layer_norm_backward(x, x, st, w, w)
    assert e.value.name == "SMC_E_OOM"
    smc.set_alloc_fail_after(0)
    assert all(torch.equal(a, b) for a, b in zip(smc.attention_backward(dout, q, k, v, out, lse, o), ref))


def test_transformer_block_over_voxels():
    """Norm, qkv by a k = 1 conv, rotary positions from the voxel coordinates,
    attention within each item, and a k = 1 conv with the residual, in fp32;
    then its input gradient through the same entry points, against the formula
    in 64 bits with torch's own derivatives."""
    from submanifold_sparse_convolution_packed_b200 import synth as S
    w = S.workload("shell2")
    keep = torch.from_numpy(w.coords[::40].copy()).cuda()
    coords = keep[torch.sort(keep[:, 0], stable=True).indices].contiguous()
    m = smc.build_map(coords, w.grid, batch=2)
    n, h, d = coords.shape[0], 4, 16
    c = h * d
    g = gen(40)
    x, dy = normal(g, n, c), normal(g, n, c)
    gamma, beta = normal(g, c, scale=0.1, shift=1.0), normal(g, c, scale=0.1)
    w1, w2 = normal(g, 3 * c, c, scale=c ** -0.5), normal(g, c, c, scale=c ** -0.5)
    o = torch.searchsorted(coords[:, 0].contiguous(), torch.arange(3, dtype=torch.int32, device="cuda"), out_int32=True)
    freqs, _ = smc.rotary_freqs(2, 3, device="cuda")
    pos = coords[:, 1:]

    def lin(a, wt):
        return smc.conv(m, a, wt.view(wt.shape[0], 1, 1, 1, wt.shape[1]), ksize=1)

    st, lse = torch.empty(n, 2, device="cuda"), torch.empty(n, h, device="cuda")
    xn = smc.layer_norm(x, gamma, beta, stats=st)
    qkv = lin(xn, w1).view(n, 3, h, d)
    qk = qkv[:, :2].reshape(n, 2 * h, d)
    turned = smc.rotary(qk, pos, freqs).view(n, 2, h, d)
    a = smc.attention(turned[:, 0], turned[:, 1], qkv[:, 2], o, lse=lse)
    y = smc.conv(m, a.view(n, c), w2.view(c, 1, 1, 1, c), ksize=1, residual=x)
    # backward
    da = lin(dy, w2.t().contiguous()).view(n, h, d)
    dqkv = torch.empty(n, 3, h, d, device="cuda")
    smc.attention_backward(da, turned[:, 0], turned[:, 1], qkv[:, 2], a, lse, o, dq=dqkv[:, 0], dk=dqkv[:, 1],
                           dv=dqkv[:, 2])
    heads = dqkv.view(n, 3 * h, d)[:, :2 * h]
    smc.rotary(heads, pos, freqs, inverse=True, out=heads)
    dxn = lin(dqkv.view(n, 3 * c), w1.t().contiguous())
    dx, dgamma, dbeta = smc.layer_norm_backward(dxn, x, st, gamma, beta)
    dx = dx + dy

    X, G, B = (t.double().requires_grad_() for t in (x, gamma, beta))
    mean = X.mean(1, keepdim=True)
    xn_ = (X - mean) / ((X - mean).square().mean(1, keepdim=True) + 1e-5).sqrt() * G + B
    qkv_ = (xn_ @ w1.double().t()).view(n, 3, h, d)
    ang = (pos.double()[:, :, None] * freqs).flatten(1)[:, None]

    def turn(t, ang):
        u, v = t[..., 0:12:2], t[..., 1:12:2]
        r = torch.stack([u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()], -1).flatten(-2)
        return torch.cat([r, t[..., 12:]], -1)

    parts = []
    for lo, hi in spans(o):
        q_, k_, v_ = turn(qkv_[lo:hi, 0], ang[lo:hi]), turn(qkv_[lo:hi, 1], ang[lo:hi]), qkv_[lo:hi, 2]
        p = torch.softmax(torch.einsum("ihd,jhd->hij", q_, k_) * d ** -0.5, -1)
        parts.append(torch.einsum("hij,jhd->ihd", p, v_))
    y_ = torch.cat(parts).reshape(n, c) @ w2.double().t() + X
    y_.backward(dy.double())
    # a chain of fp32 steps, each off by tens of ulp of its magnitudes
    for got, ref in ((y, y_.detach()), (dx, X.grad), (dgamma, G.grad), (dbeta, B.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) < 1e-5
    m.free()


def test_calls_launch_the_library():
    q, k, v, dout, o, *_ = _chain_inputs(4)
    before = smc.kernel_launches()
    smc.attention(q, k, v, o)
    assert smc.kernel_launches() > before


def test_other_device_of_tensors_is_refused():
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        smc.layer_norm(x, gamma=torch.ones(8))
    with pytest.raises(ValueError):
        smc.attention(x.view(4, 1, 8), x.view(4, 1, 8), x.view(4, 1, 8), torch.tensor([0, 4], dtype=torch.int32))

