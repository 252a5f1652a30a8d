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
