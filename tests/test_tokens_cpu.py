"""Layer norm, rotary positions and attention without a GPU: refusals of the C
ABI (made before any device work, with addresses that are never followed), of
the Python binding, and the frequencies of rotary positions."""
import ctypes
import math

import pytest
import torch

import submanifold_sparse_convolution_packed_b200 as smc
from submanifold_sparse_convolution_packed_b200 import _tokens

ARG, DTYPE, SHAPE, ALIAS, ALIGN = -1, -4, -5, -6, -11
P = ctypes.c_void_p
MB = 1 << 20


def at(k):
    """A distinct, aligned address no call may follow."""
    return P(4096 + k * 64 * MB)


def s2(row, head):
    return (ctypes.c_int64 * 2)(row, head)


def norm(x=at(0), n=8, c=16, gamma=None, beta=None, eps=1e-5, act=0, out=at(1), stats=None, dtype=0):
    return smc.lib().smc_layer_norm(x, n, c, gamma, beta, eps, act, out, stats, dtype, None)


def norm_bwd(dy=at(0), x=at(1), n=8, c=16, stats=at(2), gamma=None, beta=None, act=0, dx=at(3), dgamma=None,
             dbeta=None, dtype=0):
    return smc.lib().smc_layer_norm_backward(dy, x, n, c, stats, gamma, beta, act, dx, dgamma, dbeta, dtype, None)


def rot(x=at(0), xs=None, n=4, heads=2, dim=16, pos=at(1), ps=None, freqs=at(2), axes=1, nfreq=8, layout=0, scale=1.0,
        inverse=0, out=at(3), os=None, dtype=0):
    return smc.lib().smc_rotary(x, xs, n, heads, dim, pos, ps, freqs, axes, nfreq, layout, scale, inverse, out, os,
                                dtype, None)


def attn(q=at(0), qs=None, k=at(1), ks=None, v=at(2), vs=None, qo=at(3), ko=at(4), items=2, n=8, m=8, heads=4,
         kv_heads=2, dim=64, scale=0.125, causal=0, out=at(5), lse=None, dtype=1):
    return smc.lib().smc_attention(q, qs, k, ks, v, vs, qo, ko, items, n, m, heads, kv_heads, dim, scale, causal, out,
                                   lse, dtype, None)


def attn_bwd(dout=at(6), q=at(0), k=at(1), v=at(2), out=at(5), lse=at(7), qo=at(3), ko=at(4), items=2, n=8, m=8,
             heads=4, kv_heads=2, dim=64, scale=0.125, causal=0, dq=at(8), dqs=None, dk=at(9), dks=None, dv=at(10),
             dvs=None, dtype=1):
    return smc.lib().smc_attention_backward(dout, None, q, None, k, None, v, None, out, lse, qo, ko, items, n, m,
                                            heads, kv_heads, dim, scale, causal, dq, dqs, dk, dks, dv, dvs, dtype,
                                            None)


@pytest.mark.parametrize("code, call", [
    (ARG, dict(n=-1)), (ARG, dict(c=0)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=math.nan)), (ARG, dict(eps=math.inf)),
    (ARG, dict(act=3)), (DTYPE, dict(dtype=3)), (SHAPE, dict(c=(1 << 24) + 1)), (ARG, dict(x=None)),
    (ARG, dict(out=None)), (ALIGN, dict(x=P(4098))), (ALIGN, dict(stats=P(4096 + 500 * MB + 4))),
    (ALIAS, dict(out=P(4096 + 64))), (ALIAS, dict(gamma=at(1))), (ALIAS, dict(beta=at(1))), (ALIAS, dict(stats=at(1))),
    (ALIAS, dict(stats=at(0))),
])
def test_layer_norm_refuses(code, call):
    assert norm(**call) == code


@pytest.mark.parametrize("code, call", [
    (ARG, dict(n=-1)), (ARG, dict(c=0)), (ARG, dict(act=-1)), (DTYPE, dict(dtype=-1)), (ARG, dict(dy=None)),
    (ARG, dict(stats=None)), (ARG, dict(dx=None)), (ALIGN, dict(dy=P(4099))), (ALIGN, dict(dgamma=P(4098 + 640 * MB))),
    (ALIAS, dict(dx=at(2))), (ALIAS, dict(dgamma=at(1))), (ALIAS, dict(dgamma=at(5), dbeta=at(5))),
    (ALIAS, dict(dx=P(4096 + 4))), (ALIAS, dict(dbeta=at(3))),
])
def test_layer_norm_backward_refuses(code, call):
    assert norm_bwd(**call) == code


@pytest.mark.parametrize("code, call", [
    (ARG, dict(n=-1)), (ARG, dict(heads=0)), (ARG, dict(axes=0)), (ARG, dict(nfreq=0)), (ARG, dict(scale=math.nan)),
    (ARG, dict(scale=math.inf)), (ARG, dict(layout=2)), (ARG, dict(inverse=2)), (DTYPE, dict(dtype=5)),
    (SHAPE, dict(nfreq=9)), (SHAPE, dict(axes=3, nfreq=3)), (ARG, dict(pos=None)), (ARG, dict(freqs=None)),
    (ALIGN, dict(freqs=P(4100))), (ALIGN, dict(pos=P(4097))), (ARG, dict(xs=s2(-32, 16))), (ARG, dict(os=s2(0, 16))),
    (ARG, dict(os=s2(32, 8))), (ALIAS, dict(out=P(4096 + 64))), (ALIAS, dict(out=at(0), os=s2(64, 16))),
    (ALIAS, dict(out=at(1))), (ALIAS, dict(out=at(2))),
])
def test_rotary_refuses(code, call):
    assert rot(**call) == code


COMMON = [
    (ARG, dict(items=-1)), (ARG, dict(n=-1)), (ARG, dict(m=-1)), (ARG, dict(heads=0)), (ARG, dict(kv_heads=0)),
    (ARG, dict(dim=0)), (ARG, dict(scale=0.0)), (ARG, dict(scale=-1.0)), (ARG, dict(scale=math.nan)),
    (ARG, dict(scale=math.inf)), (ARG, dict(causal=2)), (DTYPE, dict(dtype=3)), (SHAPE, dict(heads=3)),
    (SHAPE, dict(heads=130, kv_heads=2)), (SHAPE, dict(dim=129)), (SHAPE, dict(n=1 << 31)), (SHAPE, dict(m=1 << 31)),
    (SHAPE, dict(n=1 << 30)), (ARG, dict(q=None)), (ARG, dict(k=None)), (ARG, dict(v=None)), (ARG, dict(qo=None)),
    (ARG, dict(ko=None)), (ARG, dict(out=None)), (ALIGN, dict(q=P(4097))), (ALIGN, dict(qo=P(4098 + 192 * MB))),
]


@pytest.mark.parametrize("code, call", COMMON + [
    (ARG, dict(qs=s2(-1, 64))), (ARG, dict(ks=s2(64, -64))), (ALIAS, dict(out=at(0))), (ALIAS, dict(out=at(1))),
    (ALIAS, dict(out=at(2))), (ALIAS, dict(out=at(3))), (ALIAS, dict(lse=at(5))), (ALIAS, dict(lse=at(4))),
    (ALIGN, dict(lse=P(4098 + 640 * MB))),
])
def test_attention_refuses(code, call):
    assert attn(**call) == code


@pytest.mark.parametrize("code, call", COMMON + [
    (ARG, dict(dout=None)), (ARG, dict(lse=None)), (ARG, dict(dq=None)), (ARG, dict(dk=None)), (ARG, dict(dv=None)),
    (ARG, dict(dqs=s2(128, 64))), (ARG, dict(dks=s2(0, 64))), (ALIAS, dict(dq=at(0))), (ALIAS, dict(dk=at(6))),
    (ALIAS, dict(dv=at(7))), (ALIAS, dict(dk=at(8))), (ALIAS, dict(dv=at(9))), (ALIAS, dict(dv=at(8))),
])
def test_attention_backward_refuses(code, call):
    assert attn_bwd(**call) == code


def test_attention_backward_refuses_gradients_that_overlap():
    def place(k, more):
        return P(4096 + k * 64 * MB + more)

    # dense gradients of 8 rows: dq 4096 bytes, dk and dv 2048
    assert attn_bwd(dk=place(8, 4094)) == ALIAS and attn_bwd(dv=place(9, 2046)) == ALIAS
    # views of packed rows that are half a head apart
    assert attn_bwd(dqs=s2(512, 64), dk=place(8, 64), dks=s2(512, 64)) == ALIAS
    assert attn_bwd(dks=s2(512, 64), dv=place(9, 126), dvs=s2(512, 64)) == ALIAS



def _places(p, rows, heads, dim, st):
    return {p + r * st[0] + h * st[1] + d for r in range(rows) for h in range(heads) for d in range(dim)}


# [rows, heads, dim] views of one buffer: (offset, (row stride, head stride)) of dq
# [6, 4, 8], dk and dv [5, 2, 8], in elements
GRADIENT_VIEWS = {
    "packed rows": ((0, (64, 8)), (32, (64, 8)), (48, (64, 8)), True),
    "packed rows, dk first": ((32, (64, 8)), (0, (64, 8)), (16, (64, 8)), True),
    "heads in turn": ((0, (96, 24)), (8, (96, 24)), (16, (96, 24)), True),
    "packed heads": ((0, (8, 200)), (48, (8, 200)), (88, (8, 200)), True),
    "apart as a whole": ((0, (40, 8)), (300, (24, 8)), (500, (16, 8)), True),
    "dk over the last head of dq": ((0, (64, 8)), (24, (64, 8)), (48, (64, 8)), False),
    "dv over the second head of dk": ((0, (64, 8)), (32, (64, 8)), (40, (64, 8)), False),
    "dq over dk's next row": ((48, (64, 8)), (0, (64, 8)), (16, (64, 8)), False),
    "rows of different strides that meet later": ((0, (64, 8)), (32, (48, 8)), (1000, (16, 8)), False),
    "heads that meet later": ((0, (96, 24)), (8, (96, 16)), (1000, (16, 8)), False),
    "dv in dk's rows, one place too early": ((0, (64, 8)), (32, (64, 8)), (47, (64, 8)), False),
    "heads that meet in a later row": ((0, (8, 200)), (40, (8, 200)), (88, (8, 200)), False),
}


@pytest.mark.parametrize("name", GRADIENT_VIEWS)
def test_gradients_that_share_a_place_are_refused(name):
    q, k, v, fine = GRADIENT_VIEWS[name]
    sets = [_places(o, r, h, 8, st) for (o, st), (r, h) in zip((q, k, v), ((6, 4), (5, 2), (5, 2)))]
    assert fine == (sum(map(len, sets)) == len(set.union(*sets)))  # the table itself, place by place
    if fine and torch.cuda.is_available():
        pytest.skip("a call that is not refused would follow the made-up addresses")
    for dtype, size in ((0, 4), (1, 2)):
        def where(view):
            return P(4096 + 512 * MB + view[0] * size)

        rc = attn_bwd(n=6, m=5, heads=4, kv_heads=2, dim=8, dq=where(q), dqs=s2(*q[1]), dk=where(k), dks=s2(*k[1]),
                      dv=where(v), dvs=s2(*v[1]), dtype=dtype)
        assert (rc == ALIAS) == (not fine), rc


def test_nothing_to_do_is_fine():
    assert norm(n=0, x=None, out=None) == 0
    assert norm_bwd(n=0, dy=None, x=None, stats=None, dx=None) == 0
    assert rot(n=0, x=None, out=None, pos=None) == 0
    assert attn(items=0) == 0 and attn(n=0, q=None, out=None) == 0
    assert attn_bwd(items=0) == 0
    assert attn_bwd(n=0, m=0, q=None, k=None, v=None, dout=None, out=None, lse=None, dq=None, dk=None, dv=None) == 0


def test_binding_refuses():
    x = torch.zeros(4, 8)
    st = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        smc.layer_norm(x)  # not on a CUDA device
    with pytest.raises(TypeError):
        smc.layer_norm(x.double())
    with pytest.raises(TypeError):
        smc.layer_norm(x[None])
    with pytest.raises(ValueError):
        smc.layer_norm(x, act="gelu")
    with pytest.raises(ValueError):
        smc.layer_norm(x, gamma=torch.ones(7))
    with pytest.raises(ValueError):
        smc.layer_norm(x, gamma=torch.ones(8).half())
    with pytest.raises(ValueError):
        smc.layer_norm(x, out=torch.zeros(8, 4).t())
    with pytest.raises(ValueError):
        smc.layer_norm(x, stats=torch.zeros(4, 3))
    with pytest.raises(ValueError):
        smc.layer_norm_backward(x.half(), x, st)
    with pytest.raises(ValueError):
        smc.layer_norm_backward(x, x, st.double())
    with pytest.raises(ValueError):
        smc.layer_norm_backward(x, x, st, dgamma=torch.zeros(9))
    with pytest.raises(ValueError):
        smc.layer_norm_backward(x, x, st)
    h = torch.zeros(4, 2, 16)
    pos, f = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.float64)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:3]), dict(freqs=f.float()), dict(freqs=f.expand(2, 8)),
                dict(layout="split"), dict(freqs=torch.zeros(1, 9, dtype=torch.float64)), dict(freqs=f[:, :0]),
                dict(out=h[:3]), dict()):
        with pytest.raises(ValueError):
            smc.rotary(**{"x": h, "positions": pos, "freqs": f, **bad})
    with pytest.raises(TypeError):
        smc.rotary(h[0], pos, f)
    o = torch.tensor([0, 4], dtype=torch.int32)
    for bad in (dict(k=h[:3], v=h[:3]), dict(v=h[..., :8]), dict(offsets=o.long()), dict(k_offsets=o[:1]),
                dict(scale=0.0), dict(scale=math.inf), dict(q=torch.zeros(4, 3, 16)), dict(out=h[:2]),
                dict(lse=torch.zeros(4, 3)), dict()):
        with pytest.raises(ValueError):
            smc.attention(**{"q": h, "k": h, "v": h, "offsets": o, **bad})
    with pytest.raises(TypeError):
        smc.attention(h, h.half(), h, o)
    with pytest.raises(TypeError):
        smc.attention(h.double(), h.double(), h.double(), o)
    g = dict(dout=h, q=h, k=h, v=h, out=h, lse=torch.zeros(4, 2), offsets=o)
    for bad in (dict(dout=h[:2]), dict(out=h.half()), dict(lse=torch.zeros(4)), dict(dq=h[..., ::2]), dict(dk=h[:1]),
                dict()):
        with pytest.raises(ValueError):
            smc.attention_backward(**{**g, **bad})


def test_rotary_freqs():
    f, scale = smc.rotary_freqs(8, axes=3)
    assert f.shape == (3, 8) and f.dtype == torch.float64 and scale == 1.0
    assert torch.allclose(f[1], 10000.0 ** (-torch.arange(8, dtype=torch.float64) / 8), rtol=1e-14)
    lin, _ = smc.rotary_freqs(8, factor=4.0)
    assert torch.allclose(lin * 4, f[:1], rtol=1e-14)
    ntk, _ = smc.rotary_freqs(8, factor=4.0, scaling="ntk")
    assert ntk[0, 0] == f[0, 0] and torch.allclose(ntk[0, -1] * 4, f[0, -1], rtol=1e-12)
    one, _ = smc.rotary_freqs(1, factor=4.0, scaling="ntk")
    assert one.tolist() == [[1.0]]
    yarn, scale = smc.rotary_freqs(32, factor=8.0, scaling="yarn", original=4096)
    ref, _ = smc.rotary_freqs(32)
    turns = 4096 * ref[0] / (2 * math.pi)
    ratio = ref[0] / yarn[0]
    assert torch.allclose(ratio[turns > 40], torch.ones(1, dtype=torch.float64))
    assert torch.allclose(ratio[turns < 0.7], torch.full((1,), 8.0, dtype=torch.float64))
    assert bool((ratio[1:] >= ratio[:-1] - 1e-12).all()) and abs(scale - (1 + 0.1 * math.log(8.0))) < 1e-15
    for bad in (dict(pairs=0), dict(pairs=4, axes=0), dict(pairs=4, base=1.0), dict(pairs=4, factor=0.5),
                dict(pairs=4, scaling="other"), dict(pairs=4, factor=2.0, scaling="yarn")):
        with pytest.raises(ValueError):
            smc.rotary_freqs(**bad)


def _yarn_ratio(pairs, base, factor, original):
    """By definition: pairs up to the last whole index at 32 turns or more over the
    original length (pair 0 where none is) keep their frequency, from the first at
    one turn or less it is divided by factor, a linear ramp in the index between."""
    lo = max(math.floor(pairs * math.log(original / (2 * math.pi * 32)) / math.log(base)), 0)
    hi = math.ceil(pairs * math.log(original / (2 * math.pi)) / math.log(base))
    share = [1.0 if i >= hi else max((i - lo) / (hi - lo), 0.0) for i in range(pairs)]
    return [1.0 / ((1 - s) + s / factor) for s in share]


@pytest.mark.parametrize("original", [3, 6, 100, 4096, 65_536, 131_072, 1_048_576, 3_000_000, 100_000_000])
@pytest.mark.parametrize("pairs, base, factor", [(64, 10_000.0, 8.0), (10, 10_000.0, 2.0), (1, 100.0, 4.0), (7, 500_000.0, 32.0)])
def test_rotary_freqs_yarn_by_turns(pairs, base, factor, original):
    ref, _ = smc.rotary_freqs(pairs, base=base)
    yarn, _ = smc.rotary_freqs(pairs, base=base, factor=factor, scaling="yarn", original=original)
    ratio = ref[0] / yarn[0]
    want = torch.tensor(_yarn_ratio(pairs, base, factor, original), dtype=torch.float64)
    assert torch.allclose(ratio, want, rtol=1e-12)
    turns = original * ref[0] / (2 * math.pi)
    assert bool((ratio[turns < 0.999] > factor * (1 - 1e-12)).all())
    # more than a pair's step above one turn: no longer divided in full
    assert bool((ratio[turns > 1.001 * base ** (1 / pairs)] < factor * (1 - 1e-3)).all())


def test_rotary_freqs_yarn_of_a_long_original():
    """The slowest of 64 pairs, place 63, turns 1.2, 2.4 and 19 times; the ramps run
    over the places 40 to 65, 45 to 70 and 59 to 84."""
    ref, _ = smc.rotary_freqs(64)
    for original, share in ((65_536, 23 / 25), (131_072, 18 / 25), (1_048_576, 4 / 25)):
        ratio = 1 / (1 - share + share / 8)
        yarn, _ = smc.rotary_freqs(64, factor=8.0, scaling="yarn", original=original)
        assert abs(float(ref[0, -1] / yarn[0, -1]) / ratio - 1) < 1e-12


class _StreamOf:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.mark.parametrize("call", [
    lambda s: smc.layer_norm(torch.zeros(4, 8), stream=s),
    lambda s: smc.layer_norm_backward(torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4, 2), stream=s),
    lambda s: smc.rotary(torch.zeros(4, 2, 16), torch.zeros(4, 1, dtype=torch.int32),
                         torch.zeros(1, 8, dtype=torch.float64), stream=s),
    lambda s: smc.attention(*[torch.zeros(4, 2, 16)] * 3, torch.tensor([0, 4], dtype=torch.int32), stream=s),
    lambda s: smc.attention_backward(*[torch.zeros(4, 2, 16)] * 5, torch.zeros(4, 2),
                                     torch.tensor([0, 4], dtype=torch.int32), stream=s)])
def test_stream_of_another_device_is_refused(call, monkeypatch):
    monkeypatch.setattr(_tokens, "_device_of", lambda *tensors: 0)  # as if the tensors were on cuda:0
    with pytest.raises(ValueError, match="stream"):
        call(_StreamOf(1))


@pytest.mark.parametrize("items", [(1 << 30) - (1 << 19), (1 << 31) - (1 << 21)])
def test_attention_backward_refuses_items_beyond_its_grid(items):
    """Each item may cost a block on the queries' and one on the keys' side."""
    assert attn_bwd(items=items) == SHAPE
