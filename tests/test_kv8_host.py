"""CPU checks of the FP8 key/value cache's entry points: arguments are refused
on the host, in the order null, shape, alignment, workspace, device."""
import ctypes

import pytest
import torch

from helpers import ensure_built

P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
GOOD = ctypes.c_void_p(0x10000)
ODD4, ODD2 = ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(ensure_built())
    lib.kv8_write.argtypes = [P, P, I32, I64, I64, P, I32, I32, I32, I32, I32, F32, P, P, P, P, P]
    lib.kv8_read.argtypes = [P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, I64, P, I64, P]
    lib.kv8_prefix_attention.argtypes = [P, I64, I32, I32, I32, I32, P, P, P, P, I32, I32, I32, P, I32, P, I64, I32, P,
                                         F32, F32, P, P, P, SZ, P]
    lib.kv8_prefix_attention_workspace_size.argtypes = [I32] * 7
    lib.kv8_prefix_attention_workspace_size.restype = SZ
    return lib


def device_status():
    return 0 if torch.cuda.is_available() else 5


def call(fn, names, base, **change):
    args = dict(base, **change)
    return fn(*[args[n] for n in names])


WRITE = dict(k=GOOD, v=GOOD, T=32, k_stride=1024, v_stride=1024, slots=GOOD, Hkv=8, D=128, num_pages=100, page_size=64,
             mode=0, min_scale=0.0, kc=GOOD, vc=GOOD, ks=GOOD, vs=GOOD, stream=None)
READ = dict(kc=GOOD, vc=GOOD, ks=GOOD, vs=GOOD, slots=GOOD, T=32, Hkv=8, D=128, num_pages=100, page_size=64, mode=1,
            k=GOOD, k_stride=1024, v=GOOD, v_stride=1024, stream=None)
ATTN = dict(q=GOOD, q_stride=48 * 128, B=32, Hq=48, Hkv=8, D=128, kc=GOOD, vc=GOOD, ks=GOOD, vs=GOOD, num_pages=1000,
            page_size=64, mode=0, pp=GOOD, prefix=1024, table=GOOD, ts=8, most=8, lens=GOOD, scale=0.1, cap=0.0,
            out=GOOD, lse=GOOD, ws=GOOD, nbytes=1 << 40, stream=None)

SHAPES = [dict(Hkv=0), dict(Hkv=1025), dict(D=96), dict(D=256), dict(page_size=8), dict(page_size=48),
          dict(page_size=512), dict(num_pages=0), dict(num_pages=1 << 25), dict(mode=2), dict(mode=-1)]
ROWS = [dict(T=0), dict(T=1 << 28), dict(k_stride=1016), dict(v_stride=1028), dict(v_stride=-1024)]


def test_write_refusals(lib):
    def status(**c):
        return call(lib.kv8_write, WRITE, WRITE, **c)
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert status(**{name: None}) == 1, name
    for c in SHAPES + ROWS + [dict(min_scale=-1.0), dict(min_scale=float("inf")), dict(min_scale=float("nan"))]:
        assert status(**c) == 2, c
    for name in ("k", "v", "kc", "vc"):
        assert status(**{name: ODD4}) == 3, name
    for name in ("slots", "ks", "vs"):
        assert status(**{name: ODD2}) == 3, name
    assert status(k=None, D=96) == 1 and status(D=96, k=ODD4) == 2
    if device_status():
        assert status() == 5 and status(slots=ODD4, ks=ODD4) == 5   # natural alignment is enough for these


def test_read_refusals(lib):
    def status(**c):
        return call(lib.kv8_read, READ, READ, **c)
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert status(**{name: None}) == 1, name
    for c in SHAPES + ROWS:
        assert status(**c) == 2, c
    for name in ("k", "v", "kc", "vc"):
        assert status(**{name: ODD4}) == 3, name
    if device_status():
        assert status() == 5


def test_attention_refusals(lib):
    def status(**c):
        return call(lib.kv8_prefix_attention, ATTN, ATTN, **c)
    for name in ("q", "kc", "vc", "ks", "vs", "out", "pp", "table", "lens"):
        assert status(**{name: None}) == 1, name
    nan, inf = float("nan"), float("inf")
    for c in SHAPES + [dict(B=0), dict(B=4097), dict(Hq=47), dict(Hq=0), dict(prefix=-1), dict(most=-1), dict(ts=7),
                       dict(most=1 << 26, ts=1 << 26), dict(q_stride=48 * 128 - 8), dict(q_stride=48 * 128 + 4),
                       dict(scale=nan), dict(scale=inf), dict(cap=-1.0), dict(cap=nan), dict(cap=inf)]:
        assert status(**c) == 2, c
    for name in ("q", "kc", "vc", "out", "ws"):
        assert status(**{name: ODD4}) == 3, name
    for name in ("ks", "vs", "pp", "table", "lens", "lse"):
        assert status(**{name: ODD2}) == 3, name
    need = lib.kv8_prefix_attention_workspace_size(32, 48, 8, 128, 1024, 8, 64)
    assert status(nbytes=need - 1) == 4 and status(ws=None) == 4
    if device_status():
        assert status(nbytes=need) == 5
        assert status(lse=None) == 5
        assert status(prefix=0, pp=None) == 5
        assert status(most=0, ts=0, table=None, lens=None) == 5


def test_attention_workspace_size(lib):
    size = lib.kv8_prefix_attention_workspace_size
    assert size(0, 48, 8, 128, 0, 1, 64) == 0 and size(1, 47, 8, 128, 0, 1, 64) == 0   # what the call refuses
    assert 256 < size(1, 48, 8, 128, 0, 1, 64) <= size(1, 48, 8, 128, 1024, 1, 64) <= size(64, 48, 8, 128, 1024, 1, 64)
    assert size(4096, 48, 8, 128, 1 << 20, 1 << 10, 64) < 8 << 30
    assert size(32, 48, 8, 128, 1024, 8, 64) == size(32, 48, 8, 128, 1024, 800, 64)    # lengths are read on the device


@pytest.mark.parametrize("hq,hkv,d", [(48, 8, 128), (32, 8, 128), (16, 1, 64), (28, 4, 64), (8, 8, 128), (9, 1, 128)])
def test_attention_workspace_of_the_largest_serves_the_smaller(lib, hq, hkv, d):
    """The size does not fall as the batch, the prefix or the tables grow, so one workspace serves a program whose batch
    shrinks and grows."""
    size = lib.kv8_prefix_attention_workspace_size
    for prefix in (0, 1, 500, 1024, 8192, 65536):
        sizes = [size(b, hq, hkv, d, prefix, 8, 64) for b in list(range(1, 700)) + [1000, 2000, 4095, 4096]]
        assert sizes == sorted(sizes), prefix
    for b in (1, 2, 17, 42, 43, 85, 86, 300, 4096):
        sizes = [size(b, hq, hkv, d, prefix, 8, 64) for prefix in list(range(0, 3000, 7)) + [8192, 20000, 65536, 1 << 20]]
        assert sizes == sorted(sizes), b
        sizes = [size(b, hq, hkv, d, 8192, most, 64) for most in (0, 1, 2, 100, 4096)]
        assert sizes == sorted(sizes), b
    for b in (42, 85):   # just before another pair of row tiles
        args = dict(B=b, Hq=48, Hkv=8, prefix=8192, nbytes=size(b + 1, 48, 8, 128, 8192, 8, 64))
        assert call(lib.kv8_prefix_attention, ATTN, ATTN, **args) != 4
