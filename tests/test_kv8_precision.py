"""The attention over the FP8 cache against 64 bits: keys that stand beside much
heavier ones, sequences with several query tokens, wide page tables."""
import math

import pytest
import torch

from test_kv8 import Batch, lib  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def many(b, rows, seed=0):
    """`rows` sequences over the very same keys, each with a query of its own: positive, so that the scores follow the
    keys' sums."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b.q = (1.0 + 0.05 * torch.randn(rows, b.hq, b.d, generator=gen, device="cuda")).to(torch.bfloat16)
    b.table = b.table[:1].repeat(rows, 1)
    b.lens = b.lens[:1].repeat(rows)
    b.lens_list = b.lens_list[:1] * rows
    return b


def key_at(b, i):
    """Page and offset of key i of the prefix, or of the own keys where there is no prefix."""
    pages = b.prefix_pages if b.prefix else b.table[0]
    return int(pages[i // b.page]), i % b.page


def scores_and_values(b, row):
    k, v = b.keys(row)
    q = b.q[row].double().reshape(b.hkv, -1, b.d)
    s = q @ k.transpose(1, 2) * b.scale
    # as in Batch.check: the fp32 sum of D products, q in f16, the scaling and exponent
    size = (q.abs() @ k.abs().transpose(1, 2)) * abs(b.scale)
    tiny = q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[:, None] * abs(b.scale)
    ds = size * (b.d + 8) * 2.0 ** -23 + tiny * 2.0 ** -25 + 2.0 ** -21 * s.abs()
    if b.cap:
        s = b.cap * torch.tanh(s / b.cap)
        ds = ds + 2.0 ** -20 * b.cap
    return s, ds.amax(-1, keepdim=True) + 2.0 ** -21, v


def check(b, out, lse, row, floor):
    """Values are of one sign, so the output is as large as the sum of its parts and its error is counted against
    itself: 2^-11 for the weights' rounding, twice a score's error, and `floor` for what f16's smallest numbers lose,
    which has to be small against the output's row for the bound to say anything."""
    s, ds, v = scores_and_values(b, row)
    w = torch.softmax(s, -1)
    want = w @ v
    lost = floor(w, v, row)
    assert bool((lost <= 2.0 ** -8 * want.amax(-1, keepdim=True)).all())
    tol = (2.0 ** -11 + 2 * ds) * want * 1.01 + lost + 1e-30
    o = out[row].double().reshape(want.shape)
    low, high = (x.float().to(torch.bfloat16).double() for x in (want - tol, want + tol))
    assert bool(((o >= low) & (o <= high)).all()), (row, float(((o - want) / want).abs().max()))
    z = torch.logsumexp(s, -1)
    assert bool(((lse[row].double().reshape(z.shape) - z).abs() <= ds[..., 0] + 2.0 ** -21 * (1 + z.abs())).all())


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("rows,hq,hkv,d,prefix,own,share", [
    (60, 12, 2, 128, 65536, 0, 0.996),     # the prefix on the tensor cores, many ranges of it and one
    (811, 48, 8, 64, 32768, 0, 0.998),
    (300, 8, 8, 128, 0, 6000, 0.9996),     # own keys, long pieces of them
    (300, 16, 1, 64, 0, 6000, 0.9996),
    (2, 8, 2, 128, 900, 0, 0.9999),        # a short prefix among the own keys' pieces
])
def test_light_keys_beside_a_dominant_one_without_value(lib, mode, rows, hq, hkv, d, prefix, own, share):
    """One key has nearly all of the weight and a value of zero: the output is the others' alone. A weight is rounded
    where f16 has its smallest steps to 2^-25 of the unit, and the heaviest key of its piece stands 2^8 above the
    unit at least: 2^-33 of the largest weight for each key."""
    b = many(Batch([own], prefix, hq, hkv, d, 64, mode, seed=21, q_scale=1.0), rows)
    b.v &= 0x7F
    n = prefix + own
    page, off = key_at(b, n // 3)
    if mode:   # its value's scale is like the others'
        b.vs[page, :, off] = b.vs[page, :, off - 1]
    b.v[page, :, off] = 0
    want = math.log(share / (1 - share) * n)
    for h in range(hkv):   # all of its elements alike: its score is their value times the query's sum
        scale = float(b.ks[page, h, off] if mode else b.ks[h])
        x = torch.tensor([want / math.sqrt(d) / scale])
        if mode and float(x) > 448:
            b.ks[page, h, off] *= float(x) / 448
        b.k[page, h, off] = x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).item()
    out, lse = b.run(lib)

    def floor(w, v, row):
        return w.amax(-1, keepdim=True) * v.sum(1)[:, None] * 2.0 ** -33

    for row in range(0, rows, max(1, rows // 4)):
        check(b, out, lse, row, floor)


@pytest.mark.parametrize("rows,hq,hkv,d,prefix,own,cap", [
    (60, 12, 2, 128, 4000, 0, 0.0),      # the prefix on the tensor cores, its last tile cut off
    (50, 16, 2, 64, 3840, 0, 30.0),
    (300, 8, 8, 128, 0, 1500, 0.0),      # own keys
    (40, 16, 1, 64, 0, 1500, 30.0),
    (2, 8, 2, 128, 900, 300, 0.0),       # a short prefix and own keys
    (60, 12, 2, 128, 2000, 500, 0.0),    # a tiled one and own keys
])
@pytest.mark.parametrize("apart", [-10, -15, -20, -40])
@pytest.mark.parametrize("what", ["zero rows", "large rows", "a light row of large scale", "a heavy row of small scale"])
def test_value_scales_far_apart(lib, what, apart, rows, hq, hkv, d, prefix, own, cap):
    """Per-token value scales 2^apart beside ordinary ones: what counts is the largest weight times scale among the keys
    that have a value. f16 loses 2^-25 of the unit of each such product, and the largest of a piece stands 2^8 above the
    unit, less the factor 2^6 up to which a tile is not looked at key by key."""
    b = many(Batch([own], prefix, hq, hkv, d, 64, 1, cap=cap, seed=22, q_scale=1.0), rows)
    b.v &= 0x7F
    n = prefix + own
    if what == "zero rows":      # kv8_write gives these the scale 1
        b.vs *= 2.0 ** apart
        some = [0, 1, 127, 128, 200] + list(range(333, n, 97)) + [n - 1]
    elif what == "large rows":   # ordinary keys among keys of next to no value
        b.vs *= 2.0 ** apart
        some = list(range(5, n, 70))
    else:
        some = [n // 3]
    for i in some:
        pages = b.prefix_pages if i < prefix else b.table[0]
        at = i if i < prefix else i - prefix
        page, off = int(pages[at // b.page]), at % b.page
        if what == "zero rows":
            b.v[page, :, off], b.vs[page, :, off] = 0x80 if i % 2 else 0, 1.0
        elif what == "large rows":
            b.vs[page, :, off] *= 2.0 ** -apart
        else:   # all of the key's elements alike: its score is their value times the query's sum
            sign = 1 if what == "a heavy row of small scale" else -1
            b.vs[page, :, off] *= 2.0 ** (apart * sign)
            x = 8.0 * sign / math.sqrt(d) / b.ks[page, :, off]
            b.k[page, :, off] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)[:, None]
    out, lse = b.run(lib)

    def floor(w, v, row):
        top = v.amax(-1)   # a row of kv8_write's own making has its scale times 448 for largest; here less, at most
        scale = torch.cat([b.vs[b.prefix_pages.long()].permute(1, 0, 2).reshape(hkv, -1)[:, :prefix],
                           b.vs[b.table[0][:-(-own // b.page)].long()].permute(1, 0, 2).reshape(hkv, -1)[:, :own]], 1).double()
        products = w * torch.where(top > 0, scale, 0.0)[:, None]
        dec = v / scale[..., None]
        return products.amax(-1, keepdim=True) * dec.sum(1)[:, None] * 2.0 ** -27

    for row in (0, rows - 1):
        check(b, out, lse, row, floor)


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("lens,prefix,tokens,hq,hkv,d", [
    ([40, 7, 129], 200, 4, 12, 2, 128),           # a short prefix
    ([300, 64, 65, 2] * 5, 3000, 3, 16, 2, 64),   # a tiled one
    ([90, 4], 0, 4, 8, 8, 128),
])
def test_several_query_tokens_of_a_sequence(lib, mode, lens, prefix, tokens, hq, hkv, d):
    """A sequence's last tokens as rows that share its pages, each seeing one token more than the one before."""
    b = Batch(lens, prefix, hq, hkv, d, 16, mode, seed=23)
    b.table = b.table.repeat_interleave(tokens, 0)
    b.lens_list = [max(n - tokens + 1 + i, 0) for n in lens for i in range(tokens)]
    b.lens = torch.tensor(b.lens_list, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(24)
    b.q = (1.5 * torch.randn(len(b.lens_list), hq, d, generator=gen, device="cuda")).to(torch.bfloat16)
    b.check(*b.run(lib))


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("rows,prefix,own", [(1, 0, 40), (3, 30, 20), (60, 3840, 0), (60, 3840, 30)])
def test_enormous_scores(lib, mode, rows, prefix, own, sign):
    """Scores of 1e34 of either sign: the largest of them takes all of the weight, as anywhere else."""
    d, hkv, hq = 64, 2, 16
    b = Batch([own] * rows, prefix, hq, hkv, d, 16, mode, seed=25)
    n = prefix + own
    b.q = torch.full((rows, hq, d), sign * 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    b.ks = torch.full_like(b.ks, 2.0 ** 45)
    usual, special = (0x7E, 0x70) if sign < 0 else (0x70, 0x7E)   # 448 and 128: one key of each head stands out
    b.k[:] = usual
    for row in range(rows if own else 1):
        for h in range(hkv):
            i = (7 * row + 11 * h + prefix + 3) % own + prefix if own else 5 + h
            pages = b.prefix_pages if i < prefix else b.table[row]
            at = i if i < prefix else i - prefix
            b.k[int(pages[at // 16]), h, at % 16] = special
    out, lse = b.run(lib)
    for row in range(0, rows, 7):
        k, v = b.keys(row)
        s = b.q[row].double().reshape(hkv, -1, d) @ k.transpose(1, 2) * b.scale
        assert float(s.abs().min()) > 1e33
        best = s.argmax(-1)
        want = torch.stack([v[h, best[h, 0]] for h in range(hkv)]).repeat_interleave(hq // hkv, 0)
        # one rounding of the weight times scale to f16, one of the sum to bf16
        assert bool(((out[row].double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -8)).all())
        z = s.amax(-1).reshape(-1)
        assert bool(((lse[row].double() - z).abs() <= z.abs() * (d + 8) * 2.0 ** -23).all())


@pytest.mark.parametrize("rows,hq,hkv,d,prefix,own", [(60, 12, 2, 128, 4000, 0), (300, 8, 8, 128, 0, 1500), (60, 12, 2, 64, 2000, 500)])
def test_value_scales_tiny_throughout(lib, rows, hq, hkv, d, prefix, own):
    """Values of 1e-24: scales down to 2^-92 keep everything."""
    b = many(Batch([own], prefix, hq, hkv, d, 64, 1, seed=26, q_scale=1.0), rows)
    b.v &= 0x7F
    b.vs *= 2.0 ** -80
    assert float(torch.where(torch.isfinite(b.vs), b.vs, 1.0).min()) >= 2.0 ** -92
    out, lse = b.run(lib)
    for row in (0, rows - 1):
        check(b, out, lse, row, lambda w, v, row: w.amax(-1, keepdim=True) * v.sum(1)[:, None] * 2.0 ** -27)


@pytest.mark.parametrize("every", [1, 3])
def test_many_tiles_key_by_key(lib, every):
    """A long run of tiles of one block, all or some of them with value scales far apart: the same bits in every call."""
    rows, hq, hkv, d, prefix = 230, 48, 8, 128, 12800
    b = many(Batch([0], prefix, hq, hkv, d, 64, 1, seed=27, q_scale=1.0), rows)
    assert lib.kv8_prefix_attention_plan(rows, hq, hkv, d, prefix, b.table.shape[1], 64, 1)["tiles_per_range"] >= 20
    b.v &= 0x7F
    b.vs *= 2.0 ** -12
    for i in range(0, prefix, 128 * every):
        page, off = key_at(b, i + i // 128 % 128)
        b.v[page, :, off], b.vs[page, :, off] = 0, 1.0
    out, lse = b.run(lib)

    def floor(w, v, row):   # 2^-27 of the largest weight times scale; a key's scale is its largest value / 448 or more
        return (w * v.amax(-1)[:, None]).amax(-1, keepdim=True) * 2.0 ** -27 * prefix

    for row in (0, 100, rows - 1):
        check(b, out, lse, row, floor)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        got = b.run(lib)
        differ += (got[0] != out).sum() + (got[1] != lse).sum()
    assert int(differ) == 0


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("rows,prefix,own", [(50, 6000, 0), (3, 100, 700), (40, 3000, 333)])
def test_empty_cache(lib, mode, rows, prefix, own):
    """Codes and scales of zero throughout: all keys weigh the same and there is no value."""
    b = Batch([own] * rows, prefix, 12, 2, 128, 16, mode, seed=28)
    for x in (b.k, b.v, b.ks, b.vs):
        x.zero_()
    out, lse = b.run(lib)
    assert bool((out == 0).all())
    want = math.log(prefix + own)   # fp32 exponents about the reference (under 2^7) and a sum of n weights
    assert bool(((lse.double() - want).abs() <= 2.0 ** -16).all())


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("batch,hq,hkv,d,prefix,own,page,extra", [
    (64, 32, 8, 128, 2048, 60, 64, 2048),    # tables of 131072 tokens
    (17, 16, 1, 64, 4999, 300, 16, 8192),
    (70, 16, 1, 64, 0, 60, 64, 512),
    (40, 16, 1, 128, 0, 250, 64, 512),
    (3, 48, 8, 128, 200, 17, 256, 100),
])
def test_tables_far_wider_than_the_lengths(lib, mode, batch, hq, hkv, d, prefix, own, page, extra):
    """Page tables sized for the longest context, with next to nothing in them."""
    b = Batch([own - 7 * i % own for i in range(batch)], prefix, hq, hkv, d, page, mode, seed=29, extra=extra)
    b.check(*b.run(lib))
