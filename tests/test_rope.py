"""Norms and rotation of queries and keys on the GPU against 64-bit forms: as bf16, and straight into the FP8 cache."""
import math

import numpy as np
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


BF16 = torch.bfloat16


def freqs_of(rope):
    """Radians per position, from the table's fractions of a turn (as whole numbers: exact)."""
    return [int(x) % 2 ** 64 for x in rope.turns.tolist()]


def rotate64(x, weight, positions, rope, inter, eps):
    """[T, H, D] fp64 -> (result, the sum of magnitudes of each result's terms); angles modulo a turn in whole numbers."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    turns = freqs_of(rope)
    rot = 2 * len(turns)
    frac = [[(p * f) % 2 ** 64 / 2 ** 64 for f in turns] for p in positions.tolist()]
    angle = 2 * math.pi * torch.tensor(frac, dtype=torch.float64, device=x.device)[:, None]
    cos, sin = torch.cos(angle) * rope.magnitude, torch.sin(angle) * rope.magnitude
    y, size = x.clone(), x.abs()
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * cos - b * sin, b * cos + a * sin
    size[..., i0] = size[..., i1] = (a.abs() + b.abs()) * max(1.0, abs(rope.magnitude))
    return y, size


# What fp32 leaves of a result before its rounding, relative to the sum of its terms' magnitudes: the norm's factor (a sum
# of squares of up to 256 values, at most 20 roundings deep, half of that after the root; a division, the root's two units,
# two products: 2^-24 * 18), the angle (2^-25 of half a turn, 2^-32 of a turn: under 2^-23 + 2^-29), sine and cosine (two
# units: 2^-22), the magnitude's product and the rotation's two: together below 2^-19.
FP32 = 2.0 ** -19


def assert_bf16(got, want, size, what=""):
    """Rounding is monotone: the output lies between the roundings of the ends of the interval around the exact value."""
    tol = size * FP32 + 1e-38
    low, high = ((want - tol).float().to(BF16).double(), (want + tol).float().to(BF16).double())
    got = got.double()
    assert bool(((got >= low) & (got <= high)).all()), (what, float(((got - want).abs() / tol).max()))


def inputs(t, hq, hkv, d, seed=0, fused=True, norm=True, far=100000):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(t, hq + 2 * hkv + 1, d, generator=gen, device="cuda") * 2
    x = (x * torch.exp(torch.randn(t, hq + 2 * hkv + 1, 1, generator=gen, device="cuda"))).to(BF16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (t,), generator=gen, device="cuda", dtype=torch.int32)
    w = [(1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(BF16) for _ in range(2)] if norm else [None, None]
    return q, k, v, pos, w


@pytest.mark.parametrize("t,hq,hkv,d,rot", [
    (1, 1, 0, 16, 16), (1, 48, 8, 128, 128), (3, 8, 8, 64, 32), (17, 5, 1, 80, 32), (33, 28, 4, 96, 48), (40, 7, 3, 112, 112),
    (65, 16, 1, 256, 64), (9, 3, 2, 192, 192), (300, 40, 8, 128, 64), (1000, 12, 2, 64, 64), (2, 300, 100, 32, 16),
    (2500, 48, 8, 128, 128),
])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotation(lib, t, hq, hkv, d, rot, inter, norm):
    q, k, _, pos, (qw, kw) = inputs(t, hq, hkv, d, seed=t + rot, norm=norm)
    rope = lib.rope_table(rot)
    qo, ko = lib.qk_norm_rope(q, k if hkv else None, pos, rope, qw, kw if hkv else None, eps=1e-5, interleaved=inter)
    assert_bf16(qo, *rotate64(q, qw, pos, rope, inter, 1e-5))
    if hkv:
        assert_bf16(ko, *rotate64(k, kw, pos, rope, inter, 1e-5))
    else:
        assert ko is None


@pytest.mark.parametrize("inter", [False, True])
def test_positions_far_and_negative(lib, inter):
    """Every position has its exact angle: zero (the values as they are), the largest and the least, and around them."""
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 123456789], dtype=torch.int32, device="cuda")
    q, k, *_ = inputs(8, 4, 2, 128, seed=5)
    rope = lib.rope_table(96, base=500000.0)
    qo, ko = lib.qk_norm_rope(q, k, pos, rope, interleaved=inter)
    assert_bf16(qo, *rotate64(q, None, pos, rope, inter, 0))
    assert_bf16(ko, *rotate64(k, None, pos, rope, inter, 0))
    assert torch.equal(qo[0], q[0]) and torch.equal(ko[0], k[0])
    assert torch.equal(qo[..., 96:], q[..., 96:]) and torch.equal(ko[..., 96:], k[..., 96:])


@pytest.mark.parametrize("kw", [dict(scaling="yarn", factor=32.0, original_len=4096, base=150000.0),
                                dict(scaling="wave", factor=8.0, original_len=8192), dict(scaling="linear", factor=4.0),
                                dict(inv_freq=[2.0, -0.5, 0.0, 1e-9, 6.28, 0.1, 0.2, 0.3])])
def test_scaled_tables(lib, kw):
    rope = lib.rope_table(16 if "inv_freq" in kw else 64, **kw)
    q, k, _, pos, (qw, kw_) = inputs(50, 6, 2, 64, seed=6)
    qo, ko = lib.qk_norm_rope(q, k, pos, rope, qw, kw_)
    assert_bf16(qo, *rotate64(q, qw, pos, rope, False, 1e-6))
    assert_bf16(ko, *rotate64(k, kw_, pos, rope, False, 1e-6))


def test_norm_of_one_side_only(lib):
    q, k, _, pos, (qw, kw) = inputs(40, 6, 2, 128, seed=7)
    rope = lib.rope_table(128)
    for a, b in ((qw, None), (None, kw)):
        qo, ko = lib.qk_norm_rope(q, k, pos, rope, a, b)
        assert_bf16(qo, *rotate64(q, a, pos, rope, False, 1e-6))
        assert_bf16(ko, *rotate64(k, b, pos, rope, False, 1e-6))


def test_norm_of_zero_and_tiny_and_huge_rows(lib):
    q, k, _, pos, (qw, kw) = inputs(8, 4, 1, 128, seed=8)
    q[0] = 0
    q[1] *= 1e-18
    q[2] *= 1e15
    rope = lib.rope_table(128)
    qo, _ = lib.qk_norm_rope(q, k, pos, rope, qw, kw, eps=1e-6)
    assert_bf16(qo, *rotate64(q, qw, pos, rope, False, 1e-6))
    assert bool((qo[0] == 0).all())


@pytest.mark.parametrize("t,d,rot", [(5, 128, 64), (700, 64, 64), (33, 80, 32)])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place_and_strided(lib, t, d, rot, inter):
    """Rows written over themselves, in the columns of a fused projection's output; the other columns stay."""
    q, k, v, pos, (qw, kw) = inputs(t, 12, 2, d, seed=9)
    rope = lib.rope_table(rot)
    want = lib.qk_norm_rope(q, k, pos, rope, qw, kw, interleaved=inter)
    base = q._base.clone() if q._base is not None else None
    mine = base.clone()
    q2, k2 = mine[:, :12], mine[:, 12:14]
    got = lib.qk_norm_rope(q2, k2, pos, rope, qw, kw, interleaved=inter, q_out=q2, k_out=k2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(mine[:, 14:], base[:, 14:])


@pytest.mark.parametrize("t,hq,hkv,d,rot,page,mode,skip", [
    (1, 48, 8, 128, 128, 64, 0, 0), (1, 8, 8, 64, 32, 16, 1, 0), (33, 16, 1, 128, 64, 16, 1, 3), (200, 28, 4, 64, 64, 32, 0, 7),
    (999, 40, 8, 128, 112, 128, 1, 0), (3000, 32, 8, 128, 128, 64, 0, 11),
])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_into_the_cache(lib, t, hq, hkv, d, rot, page, mode, skip, inter, norm):
    """Queries as qk_norm_rope's, values as kv8_write's, keys within half an E4M3 step of the exact ones; what no token's
    slot names stays as it was."""
    q, k, v, pos, (qw, kw) = inputs(t, hq, hkv, d, seed=t, norm=norm)
    rope = lib.rope_table(rot, scaling="linear", factor=2.0)
    pages = -(-t // page) + 2
    gen = torch.Generator(device="cuda").manual_seed(t)
    shape = (pages, hkv, page)

    def cache():
        return ([torch.randint(0, 127, (*shape, d), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2)]
                + [0.03 + 0.02 * torch.rand(shape if mode else (hkv,), generator=gen, device="cuda") for _ in range(2)])

    mine = cache()
    other = [x.clone() for x in mine]
    rng = np.random.default_rng(t)
    slots = rng.permutation(pages * page)[:t].astype(np.int32)
    for i, bad in zip(range(0, t, max(1, t // max(skip, 1))) if skip else (), [-1, pages * page, 2 ** 31 - 1, -2 ** 31] * t):
        slots[i] = bad
    slots = torch.from_numpy(slots).cuda()
    got = lib.kv8_norm_rope_write(q, k, v, pos, slots, rope, *mine, qw, kw, interleaved=inter, min_scale=1e-4)
    want, _ = lib.qk_norm_rope(q, k, pos, rope, qw, kw, interleaved=inter)
    assert torch.equal(got, want)
    lib.kv8_write(k, v, slots, *other, min_scale=1e-4)   # unrotated keys: only its values and untouched slots are compared
    assert torch.equal(mine[1], other[1]) and torch.equal(mine[3], other[3])
    ok = (slots >= 0) & (slots < pages * page)
    rows = slots[ok].long()

    def flat(x):
        return x.transpose(1, 2).reshape(pages * page, hkv, *x.shape[3:])

    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(flat(mine[0])[rest], flat(other[0])[rest])
    y, size = rotate64(k, kw, pos, rope, inter, 1e-6)
    y, noise = y[ok], size[ok] * FP32
    if mode:
        s = flat(mine[2])[rows].double()
        top = y.abs().amax(-1)
        exact = torch.clamp(top / 448, min=1e-4)
        assert bool(((s - exact).abs() <= noise.amax(-1) / 448 + exact * 2.0 ** -22).all())
        assert torch.equal(flat(mine[2])[rest], flat(other[2])[rest])
    else:
        s = mine[2].double()[None].expand(y.shape[0], -1)
        assert torch.equal(mine[2], other[2])
    s = s[..., None]
    dec = flat(mine[0])[rows].view(torch.float8_e4m3fn).double() * s
    y = y.clamp(-448 * s, 448 * s)
    # half a step: 2^-4 of the value, 2^-10 of the unit below the normal codes; and the quotient's rounding
    bound = torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20) + noise * (1 + 2.0 ** -4)
    assert bool(((dec - y).abs() <= bound).all())


@pytest.mark.parametrize("mode", [0, 1])
def test_cache_of_unrotated_rows_is_that_of_kv8_write(lib, mode):
    """At position 0 without norms keys come as they are: the same bits as kv8_write, special values among them."""
    t, h, d, page = 70, 4, 128, 16
    q, k, v, _, _ = inputs(t, 8, h, d, seed=1, norm=False)
    k[0, 0] = 0
    v[0, 0] = 0
    v[1, 1, 5] = float("inf")
    v[2, 2, 6] = float("nan")
    v[3, 3] = float("-inf")
    k[4, 0] *= 1e-30
    k[5, 1] *= 1e30
    pos = torch.zeros(t, dtype=torch.int32, device="cuda")
    slots = torch.arange(t, dtype=torch.int32, device="cuda") + 3
    caches = []
    for _ in range(2):
        c = [torch.zeros(6, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        caches.append(c + [torch.full((6, h, page) if mode else (h,), 0.05, device="cuda") for _ in range(2)])
    lib.kv8_norm_rope_write(q, k, v, pos, slots, lib.rope_table(64), *caches[0])
    lib.kv8_write(k, v, slots, *caches[1])
    for a, b in zip(*caches):
        nan = (a & 127 == 127) & (b & 127 == 127) if a.dtype == torch.uint8 else torch.zeros_like(a, dtype=torch.bool)
        assert bool(((a == b) | nan).all())   # (a NaN's sign is not part of its meaning)


def test_another_stream_and_graph(lib):
    """On a stream of its own, and captured: a replay follows positions and slots in device memory."""
    t, h, d, page = 24, 2, 128, 16
    q, k, v, pos, (qw, kw) = inputs(t, 12, h, d, seed=2)
    rope = lib.rope_table(128)
    cache = ([torch.zeros(4, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
             + [torch.zeros(4, h, page, device="cuda") for _ in range(2)])
    slots = torch.arange(t, dtype=torch.int32, device="cuda")
    want = lib.qk_norm_rope(q, k, pos, rope, qw, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [lib.qk_norm_rope(q, k, pos, rope, qw, kw, stream=side) for _ in range(10)]
    wrote = [lib.kv8_norm_rope_write(q, k, v, pos, slots, rope, *cache, qw, kw, stream=side) for _ in range(10)]
    torch.cuda.current_stream().wait_stream(side)
    for x in got:
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    for x in wrote:
        assert torch.equal(x, want[0])
    q_out, k_out = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.qk_norm_rope(q, k, pos, rope, qw, kw, q_out=q_out, k_out=k_out)
        lib.kv8_norm_rope_write(q, k, v, pos, slots, rope, *cache, qw, kw, q_out=q_out)
    for i in range(3):
        pos += 1000 * i
        slots.copy_(torch.randperm(t, device="cuda").to(torch.int32))
        graph.replay()
        again = [x.clone() for x in cache]
        a, b = lib.qk_norm_rope(q, k, pos, rope, qw, kw)
        assert torch.equal(q_out, a) and torch.equal(k_out, b)
        lib.kv8_norm_rope_write(q, k, v, pos, slots, rope, *again, qw, kw)
        assert all(torch.equal(x, y) for x, y in zip(cache, again))


def test_offsets_past_32_bits(lib):
    """Rows and slots beyond 2^31 bytes and elements."""
    t, hq, d = 20000, 900, 128   # 2.3e9 values of queries
    q = torch.zeros(t, hq, d, dtype=BF16, device="cuda")
    q[-3:] = torch.randn(3, hq, d, device="cuda").to(BF16)
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    rope = lib.rope_table(128)
    out, _ = lib.qk_norm_rope(q, None, pos, rope, q_out=q)
    small = torch.randn(3, hq, d, device="cuda").to(BF16)
    q[-3:] = small
    want, _ = lib.qk_norm_rope(small, None, pos[-3:].contiguous(), rope)
    lib.qk_norm_rope(q, None, pos, rope, q_out=q)
    assert torch.equal(q[-3:], want) and bool((q[:-3] == 0).all())
    del q, out
    h, page, pages = 8, 256, 8300
    k = torch.zeros(pages, h, page, d, dtype=torch.uint8, device="cuda")
    v, s = torch.zeros_like(k), torch.full((h,), 0.05, device="cuda")
    x = torch.randn(100, 3 * h, d, device="cuda").to(BF16)
    slots = torch.arange(100, dtype=torch.int32, device="cuda")
    p = pos[:100]
    lib.kv8_norm_rope_write(x[:, :h], x[:, h:2 * h], x[:, 2 * h:], p, slots + (pages - 1) * page, rope, k, v, s, s)
    few = [torch.zeros(1, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    lib.kv8_norm_rope_write(x[:, :h], x[:, h:2 * h], x[:, 2 * h:], p, slots, rope, *few, s, s)
    assert torch.equal(k[-1], few[0][0]) and torch.equal(v[-1], few[1][0])
    assert bool((k[:-1:97] == 0).all())


def test_outputs_stay_in_bounds(lib):
    for t, hq, hkv, d, rot in ((3, 5, 2, 80, 48), (130, 7, 1, 64, 64), (1, 1, 1, 256, 16)):
        q, k, _, pos, (qw, kw) = inputs(t, hq, hkv, d, seed=3)
        rope = lib.rope_table(rot)
        want = lib.qk_norm_rope(q, k, pos, rope, qw, kw)
        outs = []
        for h in (hq, hkv):
            buf = torch.full((t * h * d + 4096,), 7.0, dtype=BF16, device="cuda")
            outs.append((buf, buf[2048:2048 + t * h * d].view(t, h, d)))
        lib.qk_norm_rope(q, k, pos, rope, qw, kw, q_out=outs[0][1], k_out=outs[1][1])
        for (buf, x), y in zip(outs, want):
            assert torch.equal(x, y) and bool((buf[:2048] == 7).all()) and bool((buf[-2048:] == 7).all())


def test_python_checks_raise_before_a_launch(lib):
    q, k, v, pos, (qw, kw) = inputs(6, 4, 2, 64, seed=4, fused=False)
    rope = lib.rope_table(64)
    bad = [(q.float(), k, pos, rope), (q, k.float(), pos, rope), (q, k[:5], pos, rope), (q, k, pos.long(), rope),
           (q, k, pos[:5], rope), (q, k, pos, lib.RopeTable(rope.turns.int(), 1.0)), (q, k, pos.cpu(), rope),
           (q, k, pos, lib.rope_table(64, device="cpu")), (q, k, pos, lib.rope_table(96)),
           (q, k, pos, lib.RopeTable(rope.turns, float("nan")))]
    for args in bad:
        with pytest.raises((ValueError, lib.W4A8Error)):
            lib.qk_norm_rope(*args)
    for kw_ in (dict(q_weight=qw.float()), dict(k_weight=kw[:32]), dict(eps=-1.0), dict(q_out=q[:, :2]),
                dict(k_out=torch.empty_like(q)), dict(q_weight=qw.cpu())):
        with pytest.raises((ValueError, lib.W4A8Error)):
            lib.qk_norm_rope(q, k, pos, rope, **kw_)
    cache = ([torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
             + [torch.zeros(2, device="cuda") for _ in range(2)])
    slots = torch.zeros(6, dtype=torch.int32, device="cuda")
    for args in ((q, k, v[:5], pos, slots), (q, k, v, pos, slots[:5]), (q, k, v, pos, slots.long()), (q[..., :32], k, v, pos, slots)):
        with pytest.raises(ValueError):
            lib.kv8_norm_rope_write(*args, rope, *cache)
    with pytest.raises(lib.W4A8Error):
        lib.kv8_norm_rope_write(q, k, v, pos, slots, rope, *cache, min_scale=-1.0)
