"""Attention under scores of 2^26 and more, where an fp32 number has no room for anything beside them, with values of every
size: the largest score takes all of the weight, and equal ones share it."""
import math

import pytest
import torch

from helpers import ensure_built
from test_kv4 import Batch as Batch4
from test_kv8 import Batch as Batch8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


POWERS = [25, 26, 27, 28, 30, 40, 110]
SIZES = [-80, -30, -17, 0, 12, 20, 60, 100]   # of values, powers of two


def value4(b, page, h, off):
    c = torch.stack([b.v[page, h, off] & 15, b.v[page, h, off] >> 4], -1).flatten().double()
    f = b.vs[page, h, off].double()
    return c * f[0], c * f[0] + f[1]


def batch4(rows, own, sign, power, apart, who):
    """Keys of 7 of 15, values 2^apart times as large: of "all", or of "some" keys, every third."""
    d, hkv, hq = 64, 2, 16
    b = Batch4([own] * rows, hq, hkv, d, 16, seed=25)
    up = max(power - 60, 0)
    b.q = torch.full((rows, hq, d), sign * 2.0 ** (power - up), dtype=torch.bfloat16, device="cuda")
    b.k[:] = 0x77
    b.ks[..., 0], b.ks[..., 1] = 2.0 ** up / 64, 0.0
    if who == "all":
        b.vs *= 2.0 ** apart
    else:
        b.vs[:, :, ::3] *= 2.0 ** apart
    return b


@pytest.mark.parametrize("rows,own", [(1, 40), (3, 700), (40, 90)])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("power", POWERS)
def test_one_key_stands_out_of_4_bits(lib, rows, own, sign, power):
    for apart in SIZES:
        for who in ("all", "some"):
            one_of_4_bits(lib, rows, own, sign, power, apart, who)


def one_of_4_bits(lib, rows, own, sign, power, apart, who):
    b = batch4(rows, own, sign, power, apart, who)
    chosen = []
    for row in range(rows):
        for h in range(b.hkv):
            i = (7 * row + 11 * h + 3) % own
            page, off = int(b.table[row, i // 16]), i % 16
            b.k[page, h, off] = 0xFF if sign > 0 else 0x00
            chosen.append((row, h, page, off))
    out, lse = b.run(lib)
    for row, h, page, off in chosen:
        part, want = value4(b, page, h, off)
        got = out[row, h * 8:h * 8 + 8].double()
        # all of the weight on one key: f16's rounding of it times the step, the output's rounding
        tol = part.abs() * 2.0 ** -11 + want.abs() * 2.0 ** -8 + part.abs().amax() * 2.0 ** -20
        assert bool(((got - want).abs() <= tol * 1.01).all()), (apart, who)
        score = (15 if sign > 0 else 0) * 2.0 ** power / 64 * b.d * b.scale * sign
        assert bool(((lse[row, h * 8:h * 8 + 8].double() - score).abs() <= abs(score) * 2.0 ** -20 + 1e-3).all())


@pytest.mark.parametrize("rows,own", [(1, 40), (3, 700), (1, 9000), (40, 90)])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("power", POWERS)
def test_equal_scores_of_4_bits(lib, rows, own, sign, power):
    """The mean of the values: each weight's rounding is 2^-11 of it, and each product in f16 loses 2^-32 of the largest."""
    for apart in SIZES:
        equal_of_4_bits(lib, rows, own, sign, power, apart)


def equal_of_4_bits(lib, rows, own, sign, power, apart):
    b = batch4(rows, own, sign, power, apart, "some")
    out, lse = b.run(lib)
    score = 7 * 2.0 ** power / 64 * b.d * b.scale * sign
    for row in range(0, rows, 7):
        kc, kst, kl, vc, vst, vl = b.keys(row)
        want, mag = (vc * vst + vl).mean(1), (vc * vst.abs() + vl.abs()).mean(1)
        floor = torch.maximum(vst.abs(), vl.abs()).amax(1) * 2.0 ** -32 * vc.mean(1) + mag * 2.0 ** -18
        tol = mag * 2.0 ** -11 + want.abs() * 2.0 ** -8 + floor
        got = out[row].double().reshape(b.hkv, -1, b.d)
        assert bool(((got - want[:, None]).abs() <= tol[:, None] * 1.01).all()), apart
        assert bool(((lse[row].double() - score - math.log(own)).abs() <= abs(score) * 2.0 ** -20 + 1e-3).all())


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (6, 1, 128), (8, 2, 128)])
@pytest.mark.parametrize("power", [28, 40])
def test_several_tokens_of_4_bits(lib, hq, hkv, d, power):
    """Tokens of a sequence in one tile: one with such a query, its neighbours with ordinary ones, some without keys."""
    b = Batch4([100, 3, 33], hq, hkv, d, 16, seed=41, drafts=4)
    b.vs *= 2.0 ** -30
    wild = torch.arange(12, device="cuda") % 4 == 2
    b.q[wild] = (b.q[wild].double() * 2.0 ** power).to(torch.bfloat16)
    out, lse = b.run(lib)
    b.check(out, lse, every=4)   # the first token of each sequence
    for t in wild.nonzero().flatten().tolist():
        n = b.lens_list[t]
        if n == 0:
            assert bool((out[t] == 0).all())
            continue
        kc, kst, kl, vc, vst, vl = b.keys(t)
        q = b.q[t].double().reshape(hkv, -1, d)
        s = q @ (kc * kst + kl).transpose(1, 2) * b.scale
        best = s.amax(-1)
        two = s.topk(min(2, n), -1)
        err = (q.abs() @ (kc * kst.abs() + kl.abs()).transpose(1, 2) * b.scale).amax(-1) * (d + 8) * 2.0 ** -23
        clear = (two.values[..., 0] - two.values[..., -1] > 4 * err + 200) | (n == 1)   # (what another key weighs is nothing)
        v = torch.gather((vc * vst + vl)[:, None].expand(-1, s.shape[1], -1, -1), 2,
                         two.indices[..., :1, None].expand(-1, -1, 1, d))[..., 0, :]
        part = torch.gather((vc * vst).abs()[:, None].expand(-1, s.shape[1], -1, -1), 2,
                            two.indices[..., :1, None].expand(-1, -1, 1, d))[..., 0, :]
        got = out[t].double().reshape(v.shape)
        tol = part * 2.0 ** -11 + v.abs() * 2.0 ** -8 + part.amax(-1, keepdim=True) * 2.0 ** -20
        assert bool(clear.any())
        assert bool((((got - v).abs() <= tol * 1.01) | ~clear[..., None]).all())
        assert bool(((lse[t].double().reshape(best.shape) - best).abs() <= err + best.abs() * 2.0 ** -20 + 10).all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [2, 20, 50, 100, 300])   # 8, 4, 2, 1 and half a warp to join a row
def test_ordinary_rows_beside_one(lib, bits, d, rows):
    """One query head of one sequence with such scores, NaN among another's: all others keep their bits."""
    lens = [60 + i % 50 for i in range(rows)]
    b = Batch4(lens, 12, 2, d, 16, seed=44) if bits == 4 else Batch8(lens, 40, 12, 2, d, 16, 1, seed=44)
    plain, plain_lse = b.run(lib)
    b.q[1, 4] = (b.q[1, 4].double() * 2.0 ** 40).to(torch.bfloat16)
    b.q[0, 11, 5] = float("nan")
    out, lse = b.run(lib)
    same = torch.ones(rows, 12, dtype=torch.bool, device="cuda")
    same[1, 0:6] = False    # its kv head's other rows share its references' steps
    same[0, 6:12] = False
    assert torch.equal(out[same], plain[same]) and torch.equal(lse[same], plain_lse[same])
    assert bool(torch.isnan(out[0, 11]).all()) and bool(torch.isfinite(out[0, :11].float()).all())
    assert bool(torch.isfinite(out[1].float()).all()) and bool((lse[1, 4].abs() > 1e9).all())
    if bits == 4:
        kc, kst, kl, vc, vst, vl = b.keys(1)
        k, v = kc * kst + kl, vc * vst + vl
    else:
        k, v = b.keys(1)
    s = (b.q[1, 4].double() @ k[0].T) * b.scale
    best, second = s.topk(2).values.tolist()
    assert best - second > 1e6 * max(1.0, abs(best) * 2.0 ** -40)   # (so that the best key has all of the weight)
    want = v[0, s.argmax()]
    assert bool(((out[1, 4].double() - want).abs() <= want.abs() * 2.0 ** -8 + v[0].abs().amax() * 2.0 ** -20).all())
    assert abs(float(lse[1, 4]) - best) <= abs(best) * 2.0 ** -20
    again = b.run(lib)
    assert torch.equal(again[0].view(torch.int16), out.view(torch.int16)) and torch.equal(again[1][1:], lse[1:])


@pytest.mark.parametrize("rows,own", [(1, 40), (40, 90)])
def test_enormous_cap_of_4_bits(lib, rows, own):
    """Scores at both ends of a cap of 2^31 and between: equal ones at its end share the weight."""
    b = batch4(rows, own, 1, 40, 3, "some")
    b.cap = 2.0 ** 31
    b.k[:, :, ::2] = 0x00    # half of the keys score nothing
    out, lse = b.run(lib)
    for row in range(0, rows, 7):
        kc, kst, kl, vc, vst, vl = b.keys(row)
        w = (kc[..., 0] > 0).double()[..., None]
        want, mag = ((x * w).sum(1) / w.sum(1) for x in (vc * vst + vl, vc * vst.abs() + vl.abs()))
        got = out[row].double().reshape(b.hkv, -1, b.d)
        assert bool(((got - want[:, None]).abs() <= (mag * 2.0 ** -10 + want.abs() * 2.0 ** -8)[:, None] * 1.01).all())
        assert bool(((lse[row].double() / 2.0 ** 31 - 1).abs() <= 2.0 ** -20).all())


# ---------------------------------------------------------------- the FP8 cache
PREFIXES = [(1, 0, 40), (3, 30, 20), (3, 0, 700), (60, 3840, 0), (60, 3840, 30)]


def batch8(rows, prefix, own, mode, sign, power, apart, who, special):
    d, hkv, hq = 64, 2, 16
    b = Batch8([own] * rows, prefix, hq, hkv, d, 16, mode, seed=25)
    up = max(power - 60, 0)
    # a score of 128 d scale q ks in natural units
    b.q = torch.full((rows, hq, d), sign * 2.0 ** (power - up), dtype=torch.bfloat16, device="cuda")
    b.ks = torch.full_like(b.ks, 2.0 ** (up - 10))
    b.k[:] = 0x70   # 128
    if mode and who == "all":
        b.vs *= 2.0 ** apart
    elif mode:
        b.vs[:, :, ::3] *= 2.0 ** apart
    if special:
        for row in range(rows if own else 1):
            for h in range(hkv):
                i = (7 * row + 11 * h + prefix + 3) % own + prefix if own else 5 + h
                pages = b.prefix_pages if i < prefix else b.table[row]
                at = i if i < prefix else i - prefix
                b.k[int(pages[at // 16]), h, at % 16] = 0x7E if sign > 0 else 0x60   # 448, 32
    return b


@pytest.mark.parametrize("rows,prefix,own", PREFIXES)
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("power", POWERS)
def test_one_key_stands_out_of_8_bits(lib, rows, prefix, own, sign, power):
    for mode, apart, who in [(0, 0, "all")] + [(1, a, w) for a in SIZES for w in ("all", "some")]:
        one_of_8_bits(lib, rows, prefix, own, sign, power, mode, apart, who)


def one_of_8_bits(lib, rows, prefix, own, sign, power, mode, apart, who):
    b = batch8(rows, prefix, own, mode, sign, power, apart, who, True)
    out, lse = b.run(lib)
    for row in range(0, rows, 7):
        k, v = b.keys(row)
        s = b.q[row].double().reshape(b.hkv, -1, b.d) @ k.transpose(1, 2) * b.scale
        best = s.argmax(-1)
        want = torch.stack([v[h, best[h, 0]] for h in range(b.hkv)]).repeat_interleave(b.hq // b.hkv, 0)
        assert bool(((out[row].double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -8) * 1.01).all()), (mode, apart, who)
        z = s.amax(-1).reshape(-1)
        assert bool(((lse[row].double() - z).abs() <= z.abs() * 2.0 ** -20 + 1e-3).all())


@pytest.mark.parametrize("rows,prefix,own", PREFIXES)
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("power", POWERS)
def test_equal_scores_of_8_bits(lib, rows, prefix, own, sign, power):
    """The mean of the values: each weight's rounding is 2^-11 of it, and each product in f16 loses 2^-27 of the largest."""
    for mode, apart in [(0, 0)] + [(1, a) for a in SIZES]:
        equal_of_8_bits(lib, rows, prefix, own, sign, power, mode, apart)


def equal_of_8_bits(lib, rows, prefix, own, sign, power, mode, apart):
    b = batch8(rows, prefix, own, mode, sign, power, apart, "some", False)
    out, lse = b.run(lib)
    for row in range(0, rows, 7):
        k, v = b.keys(row)
        s = float((b.q[row, 0].double() @ k[0].T * b.scale).mean())
        want, mag = v.mean(1), v.abs().mean(1)
        floor = v.abs().amax() * 2.0 ** -27 + mag * 2.0 ** -18
        tol = mag * 2.0 ** -11 + want.abs() * 2.0 ** -8 + floor
        got = out[row].double().reshape(b.hkv, -1, b.d)
        assert bool(((got - want[:, None]).abs() <= tol[:, None] * 1.01).all()), apart
        assert bool(((lse[row].double() - s - math.log(k.shape[1])).abs() <= abs(s) * 2.0 ** -20 + 1e-3).all())
