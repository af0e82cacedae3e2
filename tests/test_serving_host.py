"""CPU checks of the page maps', the rotation's and the 4-bit cache's entry points: arguments are refused on the host, in
the order null, shape, alignment, workspace, device; and of the rotation's table of frequencies."""
import ctypes
import math

import pytest
import torch

import w4a8_moe_gb300 as pkg
from helpers import ensure_built

P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
GOOD = ctypes.c_void_p(0x10000)
ODD4, ODD2 = ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10002)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    return pkg._load()


def device_status():
    return 0 if torch.cuda.is_available() else 5


def refusals(fn, base, nulls, shapes, odd4, odd2, workspace=False):
    """Every refusal, and that an earlier kind goes before a later one."""
    def status(**change):
        return fn(*dict(base, **change).values())
    for name in nulls:
        assert status(**{name: None}) == 1, name
    for c in shapes:
        assert status(**c) == 2, c
        assert status(**{**c, nulls[0]: None}) == 1
        assert status(**{**c, (odd4 + odd2)[0]: ODD2}) == 2
    for name in odd4:
        assert status(**{name: ODD4}) == 3, name
    for name in odd2:
        assert status(**{name: ODD2}) == 3, name
        if not torch.cuda.is_available():
            assert status(**{name: ODD4}) == 5, name
    if workspace:
        assert status(ws=None) == 4 and status(nbytes=128) == 4
        assert status(ws=ODD4) == 3
    if not torch.cuda.is_available():
        assert status() == 5


ROPE = dict(q=GOOD, qs=1024, Hq=8, k=GOOD, ks=512, Hkv=4, T=7, D=128, pos=GOOD, turns=GOOD, rot=64, mag=1.0, inter=0, qw=GOOD,
            kw=None, eps=1e-6, qo=GOOD, qos=1024, ko=GOOD, kos=512, stream=None)
WRITE8 = dict(q=GOOD, qs=1024, Hq=8, k=GOOD, ks=512, v=GOOD, vs=512, Hkv=4, T=7, D=128, pos=GOOD, slots=GOOD, turns=GOOD, rot=64,
              mag=1.0, inter=0, qw=GOOD, kw=GOOD, eps=1e-6, pages=10, page=64, mode=1, min_scale=0.0, qo=GOOD, qos=1024, kc=GOOD,
              vc=GOOD, ksc=GOOD, vsc=GOOD, stream=None)
EXTEND = dict(lens=GOOD, new=GOOD, B=32, table=GOOD, stride=20, most=20, page=64, stack=GOOD, count=GOOD, pages=1000, cap=40,
              starts=GOOD, seqs=GOOD, positions=GOOD, seen=GOOD, slots=GOOD, out=GOOD, ws=GOOD, nbytes=256, stream=None)
TRUNCATE = dict(lens=GOOD, keep=GOOD, B=32, table=GOOD, stride=20, most=20, page=64, stack=GOOD, count=GOOD, pages=1000,
                out=GOOD, ws=GOOD, nbytes=256, stream=None)
WRITE4 = dict(k=GOOD, v=GOOD, T=32, ks=1024, vs=1024, slots=GOOD, Hkv=8, D=128, pages=100, page=64, kc=GOOD, vc=GOOD, ksc=GOOD,
              vsc=GOOD, stream=None)
READ4 = dict(kc=GOOD, vc=GOOD, ksc=GOOD, vsc=GOOD, slots=GOOD, T=32, Hkv=8, D=128, pages=100, page=64, k=GOOD, ks=1024, v=GOOD,
             vs=1024, stream=None)
ATTN4 = dict(q=GOOD, qs=48 * 128, T=32, Hq=48, Hkv=8, D=128, kc=GOOD, vc=GOOD, ksc=GOOD, vsc=GOOD, pages=1000, page=64,
             table=GOOD, stride=8, seqs_n=32, most=8, seqs=GOOD, lens=GOOD, scale=0.1, cap=0.0, out=GOOD, lse=GOOD, ws=GOOD,
             nbytes=1 << 40, stream=None)
CACHE = [dict(Hkv=0), dict(Hkv=1025), dict(D=96), dict(D=256), dict(page=8), dict(page=48), dict(page=512), dict(pages=0),
         dict(pages=1 << 25)]
POOL = [dict(B=0), dict(B=4097), dict(most=0), dict(stride=19), dict(page=8), dict(page=48), dict(page=512), dict(pages=0),
        dict(pages=1 << 25), dict(most=1 << 25, stride=1 << 25)]
TURN = [dict(T=0), dict(Hq=0), dict(rot=0), dict(rot=24), dict(rot=144), dict(qs=1016), dict(qos=1028), dict(mag=INF),
        dict(mag=NAN), dict(inter=2), dict(eps=-1.0), dict(eps=NAN)]


def test_qk_norm_rope(lib):
    refusals(lib.qk_norm_rope, ROPE, ["q", "pos", "turns", "k", "qo", "ko"],
             TURN + [dict(Hkv=-1), dict(D=120), dict(D=8), dict(D=272), dict(ks=500), dict(kos=508), dict(Hq=65532, qs=1 << 24, qos=1 << 24)],
             ["q", "k", "turns", "qw", "qo", "ko"], ["pos"])
    none = dict(ROPE, k=None, ks=0, Hkv=0, ko=None, kos=0, kw=None)
    assert lib.qk_norm_rope(*none.values()) == 5 or torch.cuda.is_available()


def test_kv8_norm_rope_write(lib):
    refusals(lib.kv8_norm_rope_write, WRITE8, ["q", "k", "v", "pos", "slots", "turns", "qo", "kc", "vc", "ksc", "vsc"],
             TURN + CACHE + [dict(ks=500), dict(vs=508), dict(mode=2), dict(min_scale=-1.0), dict(min_scale=INF), dict(T=1 << 30)],
             ["q", "k", "v", "turns", "qw", "kw", "qo", "kc", "vc"], ["pos", "slots", "ksc", "vsc"])


def test_kv_pages(lib):
    names = ["lens", "new", "table", "stack", "count", "starts", "seqs", "positions", "seen", "slots", "out"]
    refusals(lib.kv_pages_extend, EXTEND, names, POOL + [dict(cap=0), dict(cap=1 << 30)], [], names, workspace=True)
    names = ["lens", "keep", "table", "stack", "count", "out"]
    refusals(lib.kv_pages_truncate, TRUNCATE, names, POOL, [], names, workspace=True)
    assert lib.kv_pages_workspace_size() == 256


def test_kv4_write_and_read(lib):
    rows = [dict(T=0), dict(T=1 << 28), dict(ks=1016), dict(vs=1028), dict(vs=-1024)]
    names = ["k", "v", "slots", "kc", "vc", "ksc", "vsc"]
    for fn, base in ((lib.kv4_write, WRITE4), (lib.kv4_read, READ4)):
        refusals(fn, base, names, CACHE + rows, ["k", "v", "kc", "vc", "ksc", "vsc"], ["slots"])


def test_kv4_attention(lib):
    refusals(lib.kv4_attention, ATTN4, ["q", "kc", "vc", "ksc", "vsc", "table", "lens", "out"],
             CACHE + [dict(T=0), dict(T=4097), dict(Hq=47), dict(qs=48 * 128 - 8), dict(qs=48 * 128 + 4), dict(stride=7),
                      dict(most=-1), dict(most=1 << 25, stride=1 << 25), dict(seqs_n=0), dict(seqs=None, seqs_n=31),
                      dict(scale=NAN), dict(cap=-1.0), dict(cap=INF)],
             ["q", "kc", "vc", "ksc", "vsc", "out"], ["table", "seqs", "lens", "lse"], workspace=True)
    need = lib.kv4_attention_workspace_size(32, 48, 8, 128, 8, 64)
    assert lib.kv4_attention(*dict(ATTN4, nbytes=need - 1).values()) == 4
    if not torch.cuda.is_available():
        assert lib.kv4_attention(*dict(ATTN4, nbytes=need).values()) == 5
        assert lib.kv4_attention(*dict(ATTN4, most=0, stride=0, table=None, lens=None, seqs=None, seqs_n=0).values()) == 5
    sizes = [lib.kv4_attention_workspace_size(t, 48, 8, 128, 8, 64) for t in (1, 2, 33, 500, 4096)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert lib.kv4_attention_workspace_size(4097, 48, 8, 128, 8, 64) == 0
    assert lib.kv4_attention_workspace_size(32, 48, 8, 128, 1, 16) == need


# ---------------------------------------------------------------- the table of frequencies
def radians(table):
    return [(int(x) % 2 ** 64) / 2 ** 64 * 2 * math.pi for x in table.turns.tolist()]


@pytest.mark.parametrize("rot", [16, 48, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_table_plain_linear_and_base(rot, base):
    n = rot // 2
    want = [base ** (-2 * i / rot) for i in range(n)]
    plain = pkg.rope_table(rot, base=base, device="cpu")
    assert plain.magnitude == 1.0 and plain.turns.dtype == torch.int64 and plain.turns.shape == (n,)
    # two roundings of doubles each: a few 2^-53, and 2^-64 of a turn
    for got, x in zip(radians(plain), want):
        assert abs(got - x) <= x * 2.0 ** -48 + 2.0 ** -60
    half = pkg.rope_table(rot, base=base, scaling="linear", factor=2.0, device="cpu")
    for got, x in zip(radians(half), want):
        assert abs(got - x / 2) <= x * 2.0 ** -48 + 2.0 ** -60
    raised = pkg.rope_table(rot, base=base, scaling="base", factor=4.0, device="cpu")
    for i, got in enumerate(radians(raised)):
        x = (base * 4.0 ** (rot / (rot - 2))) ** (-2 * i / rot)
        assert abs(got - x) <= x * 2.0 ** -44 + 2.0 ** -60
    # the slowest pair stretches by the factor (and a table entry is 2^-64 of a turn, under 2^-61, below its number)
    assert abs(radians(raised)[-1] - want[-1] / 4) <= want[-1] * 2.0 ** -44 + 2.0 ** -60


def test_table_by_pairs_and_by_wavelength():
    plain = radians(pkg.rope_table(128, base=10000.0, device="cpu"))
    yarn = pkg.rope_table(128, scaling="yarn", factor=16.0, original_len=4096, device="cpu")
    got = radians(yarn)
    assert yarn.magnitude == pytest.approx(0.1 * math.log(16.0) + 1, rel=2.0 ** -23)
    over = [4096 * f / (2 * math.pi) for f in plain]   # turns over the original length
    for i, (f, g) in enumerate(zip(plain, got)):
        ratio = f / g
        assert 1 - 1e-12 <= ratio <= 16 + 1e-9
        if over[i] > 33 * 10000 ** (2 / 128):      # (the ramp's ends are whole pairs)
            assert ratio == pytest.approx(1, abs=1e-12)
        if over[i] < 1 / 10000 ** (2 / 128) / 1.01:
            assert ratio == pytest.approx(16, rel=1e-12)
    assert all(a / b <= c / d + 1e-9 for a, b, c, d in zip(plain, got, plain[1:], got[1:]))
    wave = radians(pkg.rope_table(128, scaling="wave", factor=8.0, original_len=8192, device="cpu"))
    for f, g in zip(plain, wave):
        r = 8192 * f / (2 * math.pi)
        keep = 1.0 if r > 4 else 0.0 if r < 1 else (r - 1) / 3
        assert g == pytest.approx(f * keep + f / 8 * (1 - keep), rel=1e-10)


def test_table_by_pairs_where_no_pair_is_between():
    """All pairs turn more than `high` times over the original length, or all of them less than `low` times."""
    for rot, base, length, low, high, ratio in ((64, 2.0, 4.0e5, 1.0, 32.0, 1), (16, 10.0, 1.0e9, 1.0, 32.0, 1),
                                                (64, 10000.0, 4.0, 1.0, 32.0, 8), (16, 100.0, 64.0, 900.0, 1000.0, 8),
                                                (128, 1.5, 2.0, 1.0, 32.0, 8)):
        plain = radians(pkg.rope_table(rot, base=base, device="cpu"))
        over = [length * f / (2 * math.pi) for f in plain]
        assert min(over) > high if ratio == 1 else max(over) < low
        got = radians(pkg.rope_table(rot, base=base, scaling="yarn", factor=8.0, original_len=length, low=low, high=high,
                                     device="cpu"))
        for f, g in zip(plain, got):
            assert f / g == pytest.approx(ratio, rel=1e-12)


def test_table_of_own_frequencies():
    own = [1.0, -0.25, 0.0, 6.25, -6.25, 1e-12, 2 * math.pi, 0.5]
    for got, x in zip(radians(pkg.rope_table(16, inv_freq=own, device="cpu")), own):
        d = (got - x) % (2 * math.pi)
        assert min(d, 2 * math.pi - d) <= 2.0 ** -48


def test_table_refusals(lib):
    for kw in (dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=272), dict(rotary_dim=0), dict(base=1.0), dict(base=NAN),
               dict(base=INF), dict(scaling="linear", factor=0.5), dict(scaling="base", factor=INF),
               dict(scaling="yarn", factor=4.0), dict(scaling="wave", factor=4.0, original_len=0.5),
               dict(scaling="wave", factor=4.0, original_len=4096, low=4.0, high=4.0),
               dict(scaling="yarn", factor=4.0, original_len=4096, low=0.0), dict(inv_freq=[7.0] + [0.0] * 31),
               dict(inv_freq=[NAN] + [0.0] * 31)):
        with pytest.raises(pkg.W4A8Error):
            pkg.rope_table(**dict(dict(rotary_dim=64, device="cpu"), **kw))
    for kw in (dict(scaling="cubic"), dict(inv_freq=[1.0]), dict(inv_freq=[1.0] * 32, scaling="linear")):
        with pytest.raises(ValueError):
            pkg.rope_table(**dict(dict(rotary_dim=64, device="cpu"), **kw))
    turns, mag = (ctypes.c_uint64 * 32)(), ctypes.c_float()
    assert lib.rope_table(64, None, 1e4, 0, 1.0, 0.0, 1.0, 2.0, None, ctypes.byref(mag)) == 1
    assert lib.rope_table(64, None, 1e4, 5, 1.0, 0.0, 1.0, 2.0, turns, ctypes.byref(mag)) == 2
