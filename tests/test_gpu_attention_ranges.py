"""Windowed and cache attention on the GPU where sizes of values are far apart: float16's exponents, infinities."""

import math

import pytest
import torch

import attention_oracle as oracle
from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, close, ints, offsets

pytestmark = [pytest.mark.gpu, needs_gpu]


def rms_close(name, got, want, u):
    """The mean square error of a gradient of independent terms. Each term is rounded once where it enters its product
    and the sum once more, either by at most u of its value and by u / sqrt(3) in the mean (an even spread over the
    step); both together sqrt(2 / 3) u = 0.82 u. float32 sums and the row's delta add less than the rest up to u."""
    got, want = got.double().cpu(), want.double().cpu()
    off = ((got - want).square().mean() / want.square().mean()).sqrt().item()
    print(f"{name}: mean error {off / u:.3f} u", flush=True)
    assert off <= u, f"{name}: mean error {off / u:.2f} u"


def gradients(m, q, k, v, dout, cu, **args):
    out, lse = m.rvq_window_attention(q, k, v, cu, **args)
    return m.rvq_window_attention_backward(dout, q, k, v, out, lse, cu, **args)


def draw(typ, lens, hq, hk, dim, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(sum(lens), h, dim, generator=g).to(TYPES[typ]).to(DEV) for h in (hq, hk, hk, hq)]


# ---------------------------------------------------------------- gradients: clips of other sizes

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 3)])
def test_a_clip_beside_a_louder_one(typ, window, sinks):
    """Gradients of a clip whose dout is 2^14 below another's in the call: those of the clip alone, bit for bit."""
    m = rvq()
    lens = [500, 700, 60]
    announce("louder clips", typ=typ, lens=lens, window=window, sinks=sinks)
    q, k, v, dout = draw(typ, lens, 2, 2, 64)
    dout[:500] *= 2.0 ** -8
    dout[500:1200] *= 2.0 ** 6
    got = gradients(m, q, k, v, dout, ints(offsets(lens)), window=window, sinks=sinks)
    for lo, hi in zip(offsets(lens), offsets(lens)[1:]):
        s = slice(lo, hi)
        alone = gradients(m, q[s], k[s], v[s], dout[s], ints([0, hi - lo]), window=window, sinks=sinks)
        for name, a, b in zip(("dq", "dk", "dv"), got, alone):
            assert torch.equal(a[s], b), (name, lo)


@pytest.mark.parametrize("dim,hq,hk,window", [(64, 2, 1, None), (128, 1, 1, 500)])
def test_float16_gradients_of_a_quiet_clip(dim, hq, hk, window):
    m = rvq()
    lens = [2000, 2000]
    announce("quiet clip", dim=dim, heads=(hq, hk), window=window)
    q, k, v, dout = draw("fp16", lens, hq, hk, dim, seed=2)
    dout[:2000] *= 2.0 ** -8
    dout[2000:] *= 2.0 ** 6
    got = gradients(m, q, k, v, dout, ints(offsets(lens)), window=window)
    s = slice(0, 2000)
    want = oracle.attention(q[s], k[s], v[s], [0, 2000], [0, 2000], window, 0, 1 / math.sqrt(dim), dout[s])
    for name, x in zip(("dq", "dk", "dv"), got):
        close(name, x[s], want[name])
        rms_close(name, x[s], want[name][0], 2.0 ** -11)


def test_float16_gradients_where_loud_frames_are_far():
    """The same within one clip: the frames from 1500 on are 2^14 louder and, by the window, do not see the first ones."""
    m = rvq()
    q, k, v, dout = draw("fp16", [2000], 1, 1, 64, seed=3)
    dout[:1500] *= 2.0 ** -8
    dout[1500:] *= 2.0 ** 6
    got = gradients(m, q, k, v, dout, ints([0, 2000]), window=200)
    want = oracle.attention(q, k, v, [0, 2000], [0, 2000], 200, 0, 1 / 8, dout)
    s = slice(0, 1000)
    for name, x in zip(("dq", "dk", "dv"), got):
        close(name, x, want[name])
        rms_close(name, x[s], want[name][0][s], 2.0 ** -11)


# ---------------------------------------------------------------- gradients: values of other sizes

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [200.0, 3000.0])
def test_float16_gradients_between_opposite_values(dim, size):
    """Two keys with equal scores and values of opposite sign: dx = dim size / 2, within float16, and larger than its
    range for a few powers of two more."""
    m = rvq()
    n = 2
    g = torch.Generator().manual_seed(5)
    q = torch.randn(n, 1, dim, generator=g).half().to(DEV)
    k = (torch.randn(1, 1, dim, generator=g) / dim).half().to(DEV).expand(n, 1, dim).contiguous()
    v = torch.tensor([size, -size], device=DEV).half().view(n, 1, 1).expand(n, 1, dim).contiguous()
    dout = torch.ones(n, 1, dim, dtype=torch.float16, device=DEV)
    announce("opposite values", dim=dim, size=size)
    got = gradients(m, q, k, v, dout, ints([0, n]))
    want = oracle.attention(q, k, v, [0, n], [0, n], None, 0, 1 / math.sqrt(dim), dout)
    for name, x in zip(("dq", "dk", "dv"), got):
        close(name, x, want[name])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(None, 0), (300, 4)])
@pytest.mark.parametrize("v_power,dout_power", [(12, -10), (15, -12), (-12, 6), (-8, 0), (0, 0)])
def test_float16_gradients_of_large_and_small_values(dim, window, sinks, v_power, dout_power):
    m = rvq()
    n = 1100
    announce("sizes of values", dim=dim, window=window, v=v_power, dout=dout_power)
    q, k, v, dout = draw("fp16", [n], 2, 1, dim, seed=6)
    v, dout = (v.clamp(-1.9, 1.9) * 2.0 ** v_power).half(), (dout * 2.0 ** dout_power).half()
    got = gradients(m, q, k, v, dout, ints([0, n]), window=window, sinks=sinks)
    want = oracle.attention(q, k, v, [0, n], [0, n], window, sinks, 1 / math.sqrt(dim), dout)
    for name, x in zip(("dq", "dk", "dv"), got):
        close(name, x, want[name])
        if want[name][0].square().mean().sqrt() > 2.0 ** -10:      # the results themselves are normal numbers
            rms_close(name, x, want[name][0], 2.0 ** -11)


def test_float16_gradients_of_sinks_and_long_clips_with_large_values():
    """Sums that are added up from pieces (queries beyond the window of the sinks, shared query heads)."""
    m = rvq()
    for lens, hq, hk, window, sinks in (([4300], 2, 1, 100, 4), ([700], 8, 1, None, 0)):
        announce("pieces", lens=lens, window=window, sinks=sinks)
        q, k, v, dout = draw("fp16", lens, hq, hk, 64, seed=7)
        v, dout = (v.clamp(-1.9, 1.9) * 2.0 ** 14).half(), (dout * 2.0 ** -12).half()
        got = gradients(m, q, k, v, dout, ints(offsets(lens)), window=window, sinks=sinks)
        want = oracle.attention(q, k, v, offsets(lens), offsets(lens), window, sinks, 1 / 8, dout)
        for name, x in zip(("dq", "dk", "dv"), got):
            close(name, x, want[name])


# ---------------------------------------------------------------- many small weights beside a large one

def sink_and_crowd(n, dim, bits):
    """One query, one key with a score `bits` powers of two above all others', whose values are 1 where its own is 0."""
    q, k, v = torch.zeros(1, 1, dim), torch.zeros(n, 1, dim), torch.ones(n, 1, dim)
    q[0, 0, 0], k[0, 0, 0] = 1.0, bits * math.log(2)
    v[0] = 0
    return q, k, v


def crowd_bound(bound, n):
    """Weights are rounded to float16 relative to their size, and below its normal numbers by half its smallest step,
    2^-25, where the largest weight stands at 2^7 or more: n of them by 2^-32 n of the largest value, here 1."""
    return bound + n * 2.0 ** -32


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bits", [14, 20, 26])
def test_small_weights_beside_a_large_one(typ, dim, bits):
    m = rvq()
    n = 40000
    announce("a sink and a crowd", typ=typ, dim=dim, bits=bits)
    q, k, v = (x.to(TYPES[typ]).to(DEV) for x in sink_and_crowd(n, dim, bits))
    for last in (False, True):                     # the large one comes first, or last
        if last:
            k, v = k.flip(0).contiguous(), v.flip(0).contiguous()
        out, lse = m.rvq_window_attention(q, k, v, ints([0, 1]), ints([0, n]), scale=1.0)
        want = oracle.attention(q, k, v, [0, 1], [0, n], None, 0, 1.0)
        close("out", out, (want["out"][0], crowd_bound(want["out"][1], n)))
        close("lse", lse, want["lse"])


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("dim,n", [(64, 40000), (128, 500)])
@pytest.mark.parametrize("bits", [14, 20, 26])
def test_small_weights_beside_a_large_one_in_a_cache(typ, dim, n, bits):
    m = rvq()
    page = 50
    announce("a sink and a crowd in a cache", typ=typ, dim=dim, n=n, bits=bits)
    q, k, v = (x.to(TYPES[typ]).to(DEV) for x in sink_and_crowd(n, dim, bits))
    pools = [x.view(n // page, page, 1, dim).transpose(1, 2).contiguous() for x in (k, v)]
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    out = m.rvq_cache_attention(q, *pools, table, ints([n]), scale=1.0)
    want = oracle.attention(q, k, v, [0, 1], [0, n], None, 0, 1.0)["out"]
    close("out", out, (want[0], crowd_bound(want[1], n)))


# ---------------------------------------------------------------- infinite values

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("dim", [64, 128])
def test_seen_infinities_keep_their_sign(typ, dim):
    """A value that is seen is infinite: so is the result, with its sign; NaN for infinities of both signs or a NaN;
    all other results as with a 0 in its place."""
    m = rvq()
    n, window, sinks = 260, 50, 2
    announce("infinite values", typ=typ, dim=dim)
    q, k, v, _ = draw(typ, [n], 2, 1, dim, seed=8)
    marks = {(0, 3): math.inf, (37, 5): math.inf, (40, 5): -math.inf, (100, 6): math.nan, (150, dim - 1): -math.inf,
             (151, 33): math.inf, (259, 0): -math.inf, (200, 8): math.inf, (202, 8): math.inf}
    bad = v.clone()
    for (j, d), x in marks.items():
        v[j, 0, d], bad[j, 0, d] = 0, x
    cu = ints([0, n])
    clean, lse = m.rvq_window_attention(q, k, v, cu, window=window, sinks=sinks)
    got, got_lse = m.rvq_window_attention(q, k, bad, cu, window=window, sinks=sinks)
    sees, want = oracle.sees(n, n, window, sinks).to(DEV), clean.clone()
    for d in {d for _, d in marks}:
        for p in range(n):
            seen = [x for (j, e), x in marks.items() if e == d and sees[p, j]]
            if seen:
                want[p, :, d] = sum(seen)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=5.0, posinf=math.inf, neginf=-math.inf), want.nan_to_num(nan=5.0, posinf=math.inf, neginf=-math.inf))
    assert torch.equal(lse, got_lse)
