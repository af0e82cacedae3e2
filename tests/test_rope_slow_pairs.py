"""Pairs that turn very slowly: their sine, next to zero, keeps all the digits of the angle."""
import math

import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


def angles(rope, positions):
    """[T, pairs] fp64: the angles within half a turn, from whole numbers, so that small ones are exact to 2^-53 of themselves."""
    turns = [int(f) % 2 ** 64 for f in rope.turns.tolist()]
    part = [[((p * f + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2 ** 64 for f in turns] for p in positions.tolist()]
    return 2 * math.pi * torch.tensor(part, dtype=torch.float64, device="cuda")


TABLES = [dict(base=500000.0, scaling="wave", factor=8.0, original_len=8192), dict(base=1e8, scaling="linear", factor=64.0),
          dict(inv_freq=[2.0 ** -i * 1.1 for i in range(1, 65)])]


@pytest.mark.parametrize("table", TABLES)
@pytest.mark.parametrize("inter", [False, True])
def test_small_angles_keep_their_digits(lib, table, inter):
    """Of each pair one value is 1 and the other 0, so that the results are the cosine and the sine alone. What is wrong
    before the rounding to bf16, relative to each of them: the angle's conversion to fp32 (2^-24), the sine (two units,
    2^-22), a product with the magnitude and one with the value (2^-24 each): together below 2^-21."""
    d = 128
    rope = lib.rope_table(d, **table)
    pos = torch.tensor([0, 1, -1, 2, 3, 7, -100, 4097, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    x = torch.zeros(len(pos), 2, d, dtype=BF16, device="cuda")
    first, second = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, d // 2), slice(d // 2, d))
    x[:, 0, first] = 1
    x[:, 1, second] = 1
    angle = angles(rope, pos)
    want = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    want[:, 0, first], want[:, 0, second] = torch.cos(angle), torch.sin(angle)
    want[:, 1, first], want[:, 1, second] = -torch.sin(angle), torch.cos(angle)
    want *= rope.magnitude
    tol = want.abs() * 2.0 ** -21 + 1e-38
    low, high = ((want - tol).float().to(BF16).double(), (want + tol).float().to(BF16).double())
    got, none = lib.qk_norm_rope(x, None, pos, rope, interleaved=inter)
    assert none is None
    assert bool(((got.double() >= low) & (got.double() <= high)).all()), float(((got.double() - want).abs() / tol).max())


def test_into_the_cache(lib):
    """The keys in the FP8 cache likewise: codes of a row's sine alone."""
    d, t = 64, 40
    rope = lib.rope_table(d, base=1e8, scaling="linear", factor=64.0)
    pos = torch.arange(1, t + 1, dtype=torch.int32, device="cuda")
    k = torch.zeros(t, d // 2, d, dtype=BF16, device="cuda")
    for i in range(d // 2):   # head i holds pair i's second value alone: its first becomes minus the sine
        k[:, i, d // 2 + i] = 1
    q = torch.zeros(t, 1, d, dtype=BF16, device="cuda")
    cache = ([torch.zeros(3, d // 2, 16, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
             + [torch.zeros(d // 2, device="cuda") for _ in range(2)])
    # scales of each head: the first token's sine is 2^-3 of the scale, the cosines saturate
    sines = torch.sin(angles(rope, pos))
    scale = sines[0].abs().float() * 8
    cache[2].copy_(scale)
    cache[3].fill_(1.0)
    lib.kv8_norm_rope_write(q, k, k, pos, torch.arange(t, dtype=torch.int32, device="cuda"), rope, *cache)
    rows = cache[0].transpose(1, 2).reshape(48, d // 2, d)[:t].view(torch.float8_e4m3fn).double() * scale.double()[:, None]
    got = rows[:, range(d // 2), range(d // 2)]
    exact = -torch.clamp(sines, -448 * scale.double(), 448 * scale.double())
    # half a step of E4M3: 2^-4 of the value; the quotient's rounding and the sine's 2^-21
    bound = exact.abs() * (2.0 ** -4 + 2.0 ** -18)
    assert bool(((got - exact).abs() <= bound).all())
    # and the code is the one of the exact quotient wherever that lies clear of a border between two
    q8 = (exact / scale.double()).float()
    clear = (q8 * (1 - 2.0 ** -19)).to(torch.float8_e4m3fn).float() == (q8 * (1 + 2.0 ** -19)).to(torch.float8_e4m3fn).float()
    assert bool((got == q8.to(torch.float8_e4m3fn).double() * scale.double())[clear].all())
