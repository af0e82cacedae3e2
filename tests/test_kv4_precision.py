"""The 4-bit cache's attention where weights, scores or values are far apart or out of the ordinary, against 64-bit forms."""
import math

import pytest
import torch

from helpers import ensure_built
from test_kv4 import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


def slot_of(b, row, i):
    return int(b.table[row, i // b.page]), i % b.page


SHAPES = [(1, 8, 8, 128, 3000), (40, 32, 8, 128, 500), (2, 16, 1, 64, 20000), (3, 9, 1, 128, 700)]


@pytest.mark.parametrize("rows,hq,hkv,d,own", SHAPES)
@pytest.mark.parametrize("share", [0.9, 0.999, 0.99999])
def test_light_keys_beside_a_dominant_one_without_value(lib, rows, hq, hkv, d, own, share):
    """One key has nearly all of the weight and a value of zero, or one value throughout: the others still add up right."""
    for least in (0.0, 2.5):
        b = Batch([own] * rows, hq, hkv, d, 64, seed=21, q_scale=1.0)
        b.q = b.q.abs()   # so that a key of equal elements scores its element times the query's sum
        for row in range(rows):
            page, off = slot_of(b, row, own // 3 + row)
            b.vs[page, :, off, 0], b.vs[page, :, off, 1] = 0, least
            b.ks[page, :, off, 0] = 0
            # about log(share / (1 - share) n) above the others
            b.ks[page, :, off, 1] = (math.log(share / (1 - share) * own) + 2) / (0.8 * d * d ** -0.5)
        b.check(*b.run(lib), every=max(1, rows // 3))


@pytest.mark.parametrize("rows,hq,hkv,d,own", SHAPES)
@pytest.mark.parametrize("apart", [-80, -30, 20, 60])
@pytest.mark.parametrize("some", ["few", "many"])
def test_values_far_apart(lib, rows, hq, hkv, d, own, apart, some):
    """Values 2^apart times as large beside ordinary ones. What counts is the largest weight times a value's size."""
    b = Batch([own] * rows, hq, hkv, d, 64, seed=22, q_scale=1.0)
    every = 97 if some == "few" else 3
    for row in range(rows):
        for i in range(row % 5, own, every):
            page, off = slot_of(b, row, i)
            b.vs[page, :, off] *= 2.0 ** apart
    b.check(*b.run(lib), every=max(1, rows // 3))


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("rows,own", [(1, 40), (3, 700), (40, 90)])
@pytest.mark.parametrize("power", [24, 26, 27, 28, 30, 110])
def test_enormous_scores(lib, rows, own, sign, power):
    """Scores of 2^power and more of either sign: the largest of them takes all of the weight, as anywhere else."""
    d, hkv, hq = 64, 2, 16
    b = Batch([own] * rows, hq, hkv, d, 16, seed=25)
    up = max(power - 60, 0)
    b.q = torch.full((rows, hq, d), sign * 2.0 ** (power - up), dtype=torch.bfloat16, device="cuda")
    b.k[:] = 0x77            # 7 of 15
    b.ks[..., 0], b.ks[..., 1] = 2.0 ** up / 64, 0.0
    chosen = []
    for row in range(rows):
        for h in range(hkv):
            i = (7 * row + 11 * h + 3) % own
            page, off = slot_of(b, row, i)
            b.k[page, h, off] = 0xFF if sign > 0 else 0x00
            chosen.append((row, h, page, off))
    out, lse = b.run(lib)
    for row, h, page, off in chosen:
        c = torch.stack([b.v[page, h, off] & 15, b.v[page, h, off] >> 4], -1).flatten().double()
        f = b.vs[page, h, off].double()
        want = c * f[0] + f[1]
        got = out[row, h * 8:h * 8 + 8].double()
        # all of the weight on one key: f16's rounding of it, the output's
        tol = (c * f[0]).abs() * 2.0 ** -11 + want.abs() * 2.0 ** -8 + 1e-30
        assert bool(((got - want).abs() <= tol * 1.01 + (c * f[0]).abs().amax() * 2.0 ** -11).all())
        score = (15 if sign > 0 else 0) * 2.0 ** power / 64 * d * b.scale * sign
        assert bool(((lse[row, h * 8:h * 8 + 8].double() - score).abs() <= abs(score) * 2.0 ** -20 + 1e-3).all())


@pytest.mark.parametrize("rows,hq,hkv,d,own", SHAPES)
def test_values_tiny_throughout(lib, rows, hq, hkv, d, own):
    """Values of 1e-24."""
    b = Batch([own] * rows, hq, hkv, d, 64, seed=26, q_scale=1.0)
    b.vs *= 2.0 ** -80
    b.check(*b.run(lib), every=max(1, rows // 3))


@pytest.mark.parametrize("rows,own", [(1, 40), (3, 5000), (60, 90)])
def test_empty_cache(lib, rows, own):
    """Codes, steps and least values of zero throughout: all keys weigh the same and there is no value."""
    b = Batch([own] * rows, 12, 2, 128, 16, seed=28)
    for x in (b.k, b.v, b.ks, b.vs):
        x.zero_()
    out, lse = b.run(lib)
    assert bool((out == 0).all())
    # fp32 exponents about the reference (under 2^7) and a sum of n weights
    assert bool(((lse.double() - math.log(own)).abs() <= 2.0 ** -16).all())
