"""Rotary positions far out on the GPU against angles of 60 decimal digits: what a float64 product of position and
frequency loses there (2^-53 of 2^30 turns are 2^-23 of one) counts too.

Bounds as in test_gpu_rotary without its part for the angle: sine and cosine are off by 6 f of the amplitude, f = 2^-24,
two products and a sum by f each, the result is rounded once.
"""

import math
from decimal import Decimal, getcontext

import pytest
import torch

from gpu_util import DEV, announce, needs_gpu, rvq
from test_gpu_attention import TYPES, ints
from test_gpu_rotary import F32, make

pytestmark = [pytest.mark.gpu, needs_gpu]

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")


def angles(positions, frequencies):
    """The angles less their whole turns, [T, n] float64."""
    getcontext().prec = 60
    rows = []
    for p in positions:
        turns = [Decimal(p) * Decimal(f) / TWO_PI for f in frequencies]
        rows.append([float((t - t.to_integral_value()) * TWO_PI) for t in turns])
    return torch.tensor(rows, dtype=torch.float64)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("top", [1.0, 3.0, 6.0])
@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, True)])
def test_far_positions_lose_nothing(typ, top, interleaved, inverse):
    m = rvq()
    announce("rotary, far", typ=typ, top=top)
    at = [0, 1, -1, 1_000_003, 2 ** 24 + 1, 2 ** 29 + 7, -2 ** 30 - 5, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, -2 ** 31 + 1]
    at += [2 ** 31 - 1 - 7919 * i for i in range(1, 20)]
    f = top * (0.5 + 0.5 * torch.rand(32, dtype=torch.float64, generator=torch.Generator().manual_seed(3)))
    q, k = make(typ, len(at), 3, 1, 64)
    got = m.rvq_rotary(q, k, f.to(DEV), positions=ints(at), interleaved=interleaved, inverse=inverse)
    torch.cuda.synchronize()
    angle, way, u = angles(at, f.tolist())[:, None], -1 if inverse else 1, torch.finfo(TYPES[typ]).eps / 2
    c, s = torch.cos(angle), torch.sin(angle) * way
    one, two = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    for x, y in zip((q, k), got):
        x, y = x.double().cpu(), y.double().cpu()
        a, b = x[..., one], x[..., two]
        for part, value in ((one, a * c - b * s), (two, b * c + a * s)):
            off = (a.abs() + b.abs()) * 8 * F32
            bound = off + u * (value.abs() + off) + F32 * value.abs() + math.ldexp(1.0, -25) * (typ == "fp16")
            over = ((y[..., part] - value).abs() / bound).max().item()
            print(f"{over:.3f} of the bound", flush=True)
            assert over <= 1
