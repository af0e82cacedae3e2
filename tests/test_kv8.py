"""The FP8 key/value cache on the GPU against plain 64-bit forms: writing,
reading back, and decode attention over a shared prefix."""
import numpy as np
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu

W4A8_ERR_INDEX = 8


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


# ---------------------------------------------------------------- references
def e4m3_table():
    vals = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        vals[c] = (-1 if c & 128 else 1) * (np.nan if c & 127 == 127 else v)
    return vals


TABLE = e4m3_table()


def encode(x):
    """fp32 values -> E4M3 codes, nearest even, saturating; by searching the table."""
    x = np.asarray(x, np.float64)
    mags = TABLE[:127]
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), 127, code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantize(x, scale, min_scale):
    """[T, H, D] fp32 -> (codes, scales [T, H]); scale None: found per token and head, in fp32."""
    if scale is None:
        size = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
        s = np.maximum((size / np.float32(448)).astype(np.float32), np.float32(min_scale))
        s = np.where(s == 0, np.float32(1), s)
    else:
        s = np.broadcast_to(scale, x.shape[:2])
    with np.errstate(invalid="ignore"):
        y = (x / s[..., None]).astype(np.float32)
    nan_in = np.isnan(x)
    return np.where(nan_in, 127, encode(y) & np.where(nan_in, 127, 255)).astype(np.uint8), s


def codes_equal(got, want):
    """A NaN's sign bit is not part of the format's meaning."""
    nan = (want & 127) == 127
    return np.array_equal(got[~nan], want[~nan]) and np.all((got[nan] & 127) == 127)


def random_cache(gen, pages, h, page, d, mode, spread=0.3):
    x = torch.randn(pages, h, page, d, generator=gen, device="cuda")
    x *= torch.exp(spread * torch.randn(pages, h, page, 1, generator=gen, device="cuda"))
    if mode:
        s = x.abs().amax(-1) / 448.0
        x /= s[..., None]
    else:
        s = 0.02 + 0.05 * torch.rand(h, generator=gen, device="cuda")
        x /= s[:, None, None]
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


class Batch:
    """A paged cache with a shared prefix and sequences of their own lengths."""

    def __init__(self, lens, prefix, hq, hkv, d, page, mode, cap=0.0, seed=0, q_scale=1.5, spread=0.3, extra=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_list, self.prefix, self.hq, self.hkv, self.d, self.page = lens, prefix, hq, hkv, d, page
        self.mode, self.cap, self.scale = mode, cap, d ** -0.5
        b = len(lens)
        n_p = -(-prefix // page)
        need = [-(-n // page) for n in lens]
        most = max(need + [1]) + extra
        pages = n_p + sum(need) + 1
        order = torch.randperm(pages, generator=gen, device="cuda").tolist()
        self.prefix_pages = torch.tensor(order[:n_p], dtype=torch.int32, device="cuda")
        table = np.full((b, most), -1, np.int32)
        at = n_p
        self.k, self.ks = random_cache(gen, pages, hkv, page, d, mode, spread)
        self.v, self.vs = random_cache(gen, pages, hkv, page, d, mode, spread)

        def spoil(pg, first):   # what lies behind the last token is no number, nor is its scale
            self.k[pg, :, first:] = 0x7F
            self.v[pg, :, first:] = 0xFF
            if mode:
                self.ks[pg, :, first:] = float("nan")
                self.vs[pg, :, first:] = float("inf")

        for i, n in enumerate(lens):
            table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            if n % page:
                spoil(int(table[i, need[i] - 1]), n % page)
        if prefix % page:
            spoil(order[n_p - 1], prefix % page)
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = (torch.randn(b, hq, d, generator=gen, device="cuda") * q_scale).to(torch.bfloat16)

    def run(self, lib, **kw):
        args = dict(sm_scale=self.scale, logit_cap=self.cap, lse=True)
        args.update(kw)
        q = args.pop("q", self.q)
        return lib.kv8_prefix_attention(q, self.k, self.v, self.ks, self.vs, self.prefix_pages, self.prefix,
                                        self.table, self.lens, **args)

    def keys(self, b):
        """fp64 K, V [heads, keys, D] of one sequence."""
        t = torch.from_numpy(TABLE).cuda()
        out = []
        for cache, s in ((self.k, self.ks), (self.v, self.vs)):
            parts = []
            for pages, n in ((self.prefix_pages, self.prefix), (self.table[b], self.lens_list[b])):
                pg = pages[:-(-n // self.page)].long()
                x = t[cache[pg].long()]
                f = s.double()
                x = x * (f[pg][..., None] if self.mode else f[:, None, None])
                parts.append(x.permute(1, 0, 2, 3).reshape(self.hkv, -1, self.d)[:, :n])
            out.append(torch.cat(parts, 1))
        return out

    def check(self, got, lse, every=1):
        """Elementwise bounds from the arithmetic, none fitted to the outcome.
        The value that the kernel rounds to bf16 lies within `tol` of the exact
        one; rounding is monotone, so the output lies between the roundings of
        the interval's ends. A score's error: the fp32 sum of D products (2^-23 per addition of the
        sum of magnitudes), q's elements in f16 below its row's largest
        (2^-25 of it each), the scaling and exponent (2^-21 of the score's size
        plus 2^-21), the cap's tanh (2^-20 of the cap). A weight's f16 rounding: 2^-11, plus the
        tail of f16's range (2^-25 of the largest weight, for each key)."""
        assert bool(torch.isfinite(got.float()).all())
        group = self.hq // self.hkv
        for b in range(0, len(self.lens_list), every):
            n = self.prefix + self.lens_list[b]
            o, z = got[b].double(), lse[b].double()
            if n == 0:
                assert bool((o == 0).all()) and bool((z == -torch.inf).all())
                continue
            k, v = self.keys(b)
            q = self.q[b].double().reshape(self.hkv, group, self.d)
            s = q @ k.transpose(1, 2) * self.scale
            size = (q.abs() @ k.abs().transpose(1, 2)) * abs(self.scale)
            tiny = q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[:, None] * abs(self.scale)
            ds = size * (self.d + 8) * 2.0 ** -23 + tiny * 2.0 ** -25 + 2.0 ** -21 * s.abs()
            if self.cap:
                s = self.cap * torch.tanh(s / self.cap)
                ds = ds + 2.0 ** -20 * self.cap
            ds = ds.amax(-1, keepdim=True) + 2.0 ** -21
            w = torch.softmax(s, -1)
            want, mag = w @ v, w @ v.abs()
            floor = w.amax(-1, keepdim=True) * v.abs().sum(1)[:, None] * 2.0 ** -25
            tol = (2.0 ** -11 + 2 * ds) * mag * 1.01 + floor + 1e-30
            o = o.reshape(want.shape)
            low, high = (x.float().to(torch.bfloat16).double() for x in (want - tol, want + tol))
            assert bool(((o >= low) & (o <= high)).all()), (b, float(((o - want).abs() / tol).max()))
            zw = torch.logsumexp(s, -1)
            zerr = (z.reshape(zw.shape) - zw).abs()
            ztol = ds[..., 0] + 2.0 ** -21 * (1 + zw.abs())
            assert bool((zerr <= ztol).all()), (b, float((zerr / ztol).max()))


# ---------------------------------------------------------------- write and read
def _rows(t, h, d, seed, special=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=gen) * torch.exp(torch.randn(t, h, 1, generator=gen))
    if special:
        x[0, 0, :] = 0
        x[t // 2, 0, 3] = float("inf")
        x[t // 2, 0, 5] = float("-inf")
        x[t // 3, h - 1, d - 1] = float("nan")
        x[t - 1, 0, :] = 1e-38
    return x.to(torch.bfloat16)


def _check_write(lib, t, h, d, page, mode, min_scale=0.0, skip=(), fused=False, seed=0):
    pages = -(-t // page) + 2
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kc, ks = random_cache(gen, pages, h, page, d, mode)
    vc, vs = random_cache(gen, pages, h, page, d, mode)
    before = [x.cpu().numpy().copy() for x in (kc, vc, ks, vs)]
    slots = np.random.default_rng(seed).permutation(pages * page)[:t].astype(np.int32)
    for i, bad in zip(skip, [-1, pages * page, 2 ** 31 - 1, -2 ** 31] * t):
        slots[i] = bad
    k, v = _rows(t, h, d, seed + 1, special=t > 4), _rows(t, h, d, seed + 2)
    if fused:
        qkv = torch.zeros(t, 3 * h * d + 8, dtype=torch.bfloat16)
        qkv[:, 8 + h * d:8 + 2 * h * d] = k.reshape(t, -1)
        qkv[:, 8 + 2 * h * d:] = v.reshape(t, -1)
        qkv = qkv.cuda()
        kg = qkv[:, 8 + h * d:8 + 2 * h * d].unflatten(1, (h, d))
        vg = qkv[:, 8 + 2 * h * d:].unflatten(1, (h, d))
    else:
        kg, vg = k.cuda(), v.cuda()
    lib.kv8_write(kg, vg, torch.from_numpy(slots).cuda(), kc, vc, ks, vs, min_scale=min_scale)
    for x, cache, scale, old_c, old_s in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
        codes, s = quantize(x.float().numpy(), None if mode else old_s[None], min_scale)
        want_c = old_c.copy().transpose(0, 2, 1, 3).reshape(pages * page, h, d)
        ok = (slots >= 0) & (slots < pages * page)
        want_c[slots[ok]] = codes[ok]
        got_c = cache.cpu().numpy().transpose(0, 2, 1, 3).reshape(pages * page, h, d)
        assert codes_equal(got_c, want_c)
        if mode:
            want_s = old_s.copy().transpose(0, 2, 1).reshape(pages * page, h)
            want_s[slots[ok]] = s[ok]
            assert np.array_equal(scale.cpu().numpy().transpose(0, 2, 1).reshape(pages * page, h), want_s)
        else:
            assert np.array_equal(scale.cpu().numpy(), old_s)


@pytest.mark.parametrize("t,h,d,page,mode", [
    (1, 8, 128, 64, 0), (1, 1, 64, 16, 1), (7, 5, 128, 16, 1), (33, 3, 64, 32, 0), (257, 8, 128, 128, 1),
    (1000, 1, 64, 256, 1), (4099, 2, 128, 64, 0),
])
def test_write(lib, t, h, d, page, mode):
    _check_write(lib, t, h, d, page, mode)


@pytest.mark.parametrize("mode", [0, 1])
def test_write_skips_and_fused_rows(lib, mode):
    _check_write(lib, 50, 4, 128, 16, mode, skip=(0, 3, 17, 49), fused=True)
    _check_write(lib, 9, 2, 64, 32, mode, skip=tuple(range(9)), fused=True)


def test_write_min_scale(lib):
    _check_write(lib, 40, 2, 128, 32, 1, min_scale=0.01)


def test_write_scale_of_every_bf16_value(lib):
    """The scale of a row is its largest magnitude / 448 as fp32 division has it, for all finite bf16 magnitudes."""
    x = torch.zeros(0x7F80, 1, 64, dtype=torch.int16)
    x[:, 0, 17] = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16)
    x = x.view(torch.bfloat16).cuda()
    pages = 0x7F80 // 256 + 1
    kc, vc = (torch.zeros(pages, 1, 256, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, 1, 256, device="cuda") for _ in range(2))
    lib.kv8_write(x, -x, torch.arange(0x7F80, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    amax = x[:, 0, 17].float()
    want = amax / torch.full_like(amax, 448.0)
    want = torch.where(want == 0, 1.0, want)
    for s in (ks, vs):
        assert torch.equal(s.reshape(-1)[:0x7F80], want)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -7, 1 / 448, 0.05, 0.1, 0.3, 1.7, 3e-5, 1.9999999, 2.0 ** -61, 1e-30, 1e-39,
                                   2.0 ** 61, 3e37])
def test_write_code_of_every_bf16_value(lib, scale):
    """Codes are those of the fp32 quotient, for every bf16 bit pattern, whatever shares the row with it."""
    bits = np.arange(0x10000, dtype=np.uint16)
    for order in (bits, np.random.default_rng(1).permutation(bits)):
        x = torch.from_numpy(order.view(np.int16).copy()).view(torch.bfloat16).reshape(1024, 1, 64).cuda()
        kc, vc = (torch.zeros(4, 1, 256, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
        s = torch.tensor([scale], device="cuda")
        lib.kv8_write(x, x, torch.arange(1024, dtype=torch.int32, device="cuda"), kc, vc, s, s)
        q = (x.float() / s[None, None]).cpu().numpy().reshape(-1)
        want = np.where(np.isnan(q), 127, encode(q))
        for c in (kc, vc):
            assert codes_equal(c.cpu().numpy().reshape(-1), want.astype(np.uint8))


@pytest.mark.parametrize("t,h,d,page,mode", [(1, 1, 64, 16, 1), (19, 5, 128, 32, 0), (333, 8, 64, 64, 1),
                                             (2049, 2, 128, 256, 0)])
def test_read(lib, t, h, d, page, mode):
    gen = torch.Generator(device="cuda").manual_seed(t)
    pages = 5 + t // page
    kc, ks = random_cache(gen, pages, h, page, d, mode)
    vc, vs = random_cache(gen, pages, h, page, d, mode)
    kc[0] = torch.arange(h * page * d, device="cuda").reshape(h, page, d).to(torch.uint8)   # every code, NaN too
    slots = np.random.default_rng(t).integers(0, pages * page, t).astype(np.int32)          # may repeat
    slots[0] = 3
    for i, bad in zip(range(1, t, 7), [-1, pages * page, -2 ** 31] * t):
        slots[i] = bad
    wide = torch.full((t, 3, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = lib.kv8_read(kc, vc, ks, vs, torch.from_numpy(slots).cuda(), k_out=wide[:, 0], v_out=wide[:, 2])
    assert bool((wide[:, 1] == 7.0).all())
    ok = (slots >= 0) & (slots < pages * page)
    for got, cache, scale in ((k, kc, ks), (v, vc, vs)):
        got = got.float().cpu().numpy().astype(np.float64)
        rows = TABLE[cache.cpu().numpy()].transpose(0, 2, 1, 3).reshape(pages * page, h, d)
        s = scale.cpu().numpy().astype(np.float64)
        s = s.transpose(0, 2, 1).reshape(pages * page, h) if mode else np.broadcast_to(s, (pages * page, h))
        want = np.zeros((t, h, d))
        want[ok] = (rows * s[..., None])[slots[ok]]
        want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16).double().numpy()   # both roundings
        assert np.array_equal(got, want, equal_nan=True)
        assert np.all(got[~ok] == 0)


def test_write_then_read_is_within_a_quantization_step(lib):
    t, h, d, page = 100, 4, 128, 16
    x = _rows(t, h, d, 3).cuda()
    cache = [torch.zeros(8, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(8, h, page, device="cuda") for _ in range(2)]
    slots = torch.arange(t, dtype=torch.int32, device="cuda") + 5
    lib.kv8_write(x, -x, slots, *cache, *scales)
    k, v = lib.kv8_read(*cache, *scales, slots)
    assert torch.equal(k, -v)
    top = x.float().abs().amax(-1, keepdim=True)
    # E4M3 keeps 4 significant bits down to 2^-6 of its unit, here top / 448
    bound = torch.maximum(x.float().abs() * 2.0 ** -4, top / 448 * 2.0 ** -10) * 1.01
    assert bool(((k.float() - x.float()).abs() <= bound).all())


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("hq,hkv,d,page,mode", [
    (48, 8, 128, 64, 0), (32, 8, 128, 16, 1), (8, 8, 64, 32, 1), (16, 1, 64, 16, 0), (9, 1, 128, 128, 1),
    (48, 1, 128, 256, 0), (28, 4, 64, 64, 1), (34, 2, 64, 16, 1),
])
def test_attention_heads_and_pages(lib, hq, hkv, d, page, mode):
    """Every head layout, both scale forms, page sizes; lengths of zero, one, around a page and a unit."""
    lens = [0, 1, 15, 16, 17, page - 1, page, page + 1, 200, 3]
    for prefix in (0, 1, 77, 300):
        b = Batch(lens, prefix, hq, hkv, d, page, mode, seed=prefix + hq)
        b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [1, 2, 3, 5, 21, 22, 43, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_batch_over_a_prefix(lib, batch, d):
    """Few and many rows over the prefix: one row, part of a tile, several tiles."""
    lens = [(7 * i) % 50 for i in range(batch)]
    for prefix, mode in ((129, 0), (1000, 1), (2051, 0)):
        b = Batch(lens, prefix, 12, 2, d, 32, mode, seed=batch)
        b.check(*b.run(lib))


@pytest.mark.parametrize("hq,hkv,d,mode", [(2, 1, 64, 0), (3, 1, 128, 1)])
def test_attention_largest_batch(lib, hq, hkv, d, mode):
    """4096 sequences, the most a call takes (every 37th checked)."""
    lens = [(i * 7) % 40 for i in range(4096)]
    for prefix in (0, 33, 500):
        b = Batch(lens, prefix, hq, hkv, d, 16, mode, seed=20)
        b.check(*b.run(lib), every=37)


@pytest.mark.parametrize("prefix", [127, 128, 255, 256, 257, 383, 640, 4097])
def test_attention_prefix_lengths(lib, prefix):
    """Prefixes that end on, before and behind a tile of keys and a page."""
    for mode, page in ((0, 16), (1, 64), (1, 256)):
        b = Batch([5, 0, 64] * 15, prefix, 16, 2, 128, page, mode, seed=prefix)
        b.check(*b.run(lib))


@pytest.mark.parametrize("batch,hq,hkv,d,prefix,own,mode", [
    (24, 32, 8, 64, 20000, 1500, 0),    # own keys for longer than the prefix takes
    (24, 32, 8, 128, 3000, 3000, 1),
    (64, 32, 8, 64, 9000, 40, 1),       # every SM taken by the prefix, or nearly
    (900, 48, 8, 64, 300, 5, 0),        # more tiles of rows than SMs
    (300, 4, 1, 64, 1000, 3, 1),        # the lengths' sums left to the join
])
def test_attention_prefix_and_own_keys_side_by_side(lib, batch, hq, hkv, d, prefix, own, mode):
    """Every way of sharing the SMs between the prefix and the sequences' own keys."""
    b = Batch([(own + i) % (own + 1) if i % 5 == 4 else own for i in range(batch)], prefix, hq, hkv, d, 64, mode, seed=own)
    b.check(*b.run(lib))


@pytest.mark.parametrize("batch,hq,hkv,d,own,extra,mode", [
    (1, 16, 1, 128, 9000, 1, 1),     # many pieces a row, joined by eight warps
    (3, 8, 8, 64, 5000, 1, 0),
    (70, 8, 1, 64, 1500, 1, 1),      # joined by four
    (70, 12, 1, 64, 2000, 200, 0),
    (30, 28, 4, 128, 1000, 1, 1),    # by two
    (70, 16, 1, 128, 900, 200, 1),   # tables wide enough for the form of 16 rows with more blocks an SM
    (70, 16, 1, 128, 900, 1, 0),     # and not
    (260, 6, 2, 128, 70, 1, 0),      # four units a warp
])
def test_attention_own_keys_alone(lib, batch, hq, hkv, d, own, extra, mode):
    """Every way of cutting the sequences' own keys into pieces and of joining them."""
    lens = [own - 37 * i % own if i % 6 != 5 else i % 3 for i in range(batch)]
    b = Batch(lens, 0, hq, hkv, d, 64, mode, seed=own, extra=extra)
    b.check(*b.run(lib))


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("batch", [2, 40])
def test_attention_logit_cap(lib, mode, batch):
    """Capped scores, from far below the cap to far above it."""
    for q_scale in (0.1, 1.5, 30.0):
        b = Batch([33 + i for i in range(batch)], 500, 48, 8, 128, 64, mode, cap=30.0, seed=4, q_scale=q_scale)
        b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [1, 64])
def test_attention_peaked_and_flat(lib, batch):
    """Scores spread over hundreds (one key wins) and all equal (the mean of the values)."""
    for q_scale in (40.0, 0.0):
        b = Batch([100] * batch, 900, 16, 2, 128, 32, 0, seed=8, q_scale=q_scale)
        b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [1, 64])
def test_attention_scales_far_apart(lib, batch):
    """Per-token scales over many binades, rising along the keys and tiny throughout."""
    b = Batch([300] * batch, 700, 16, 2, 128, 32, 1, seed=9, spread=1.5, q_scale=0.3)
    b.check(*b.run(lib))
    b.vs *= 2.0 ** -60
    b.ks *= 2.0 ** 20
    b.scale *= 2.0 ** -20
    b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [2, 50])
def test_attention_small_and_large_queries(lib, batch):
    """q outside f16's range, with sm_scale taking it back; a negative sm_scale."""
    for mul in (2.0 ** 100, 2.0 ** -100):
        b = Batch([40] * batch, 200, 12, 2, 128, 32, 0, seed=10)
        b.q = (b.q.double() * mul).to(torch.bfloat16)
        b.scale /= mul
        b.check(*b.run(lib))
    b = Batch([40] * batch, 200, 12, 2, 128, 32, 1, seed=10)
    b.scale = -b.scale
    b.check(*b.run(lib))


def test_attention_strided_queries_and_tables(lib):
    """q as columns of a fused projection, the page table as columns of a larger one."""
    b = Batch([30, 0, 70, 9], 100, 12, 2, 64, 16, 0, seed=11)
    want = b.run(lib)
    qkv = torch.randn(4, 12 * 64 + 256, device="cuda").to(torch.bfloat16)
    qkv[:, 128:128 + 12 * 64] = b.q.reshape(4, -1)
    big = torch.full((4, b.table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    big[:, 3:3 + b.table.shape[1]] = b.table
    b.table = big[:, 3:3 + b.table.shape[1]]
    got = b.run(lib, q=qkv[:, 128:128 + 12 * 64].unflatten(1, (12, 64)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_same_bits_each_call_and_any_workspace_contents(lib):
    for batch in (3, 60):
        b = Batch([3 * i for i in range(batch)], 777, 48, 8, 128, 64, 1, seed=12)
        size = lib.kv8_prefix_attention_workspace_size(batch, 48, 8, 128, 777, b.table.shape[1], 64)
        first = b.run(lib)
        for fill in (0x00, 0x7F, 0xFF):
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            ws[:256] = 0
            got = b.run(lib, ws=ws)
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
            assert lib.w4a8_device_error(ws) == 0


@pytest.mark.parametrize("batch,hq,hkv,d,prefix,own,mode", [
    (24, 32, 8, 128, 3000, 3000, 1), (200, 48, 8, 128, 2048, 300, 0), (64, 32, 8, 64, 8192, 40, 1),
])
def test_attention_same_bits_over_many_calls(lib, batch, hq, hkv, d, prefix, own, mode):
    """Copies land in another order each time; the result stays the same."""
    b = Batch([own] * batch, prefix, hq, hkv, d, 64, mode, seed=own)
    first = b.run(lib)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        got = b.run(lib)
        differ += (got[0] != first[0]).sum() + (got[1] != first[1]).sum()
    assert int(differ) == 0
    b.check(*first)


def test_attention_without_lse_and_without_own_tokens(lib):
    b = Batch([0, 0, 0], 65, 8, 2, 64, 16, 0, seed=13)
    out, lse = b.run(lib)
    b.check(out, lse)
    only, none = b.run(lib, lse=None)
    assert none is None and torch.equal(only, out)
    b.table = b.table[:, :0]
    got = b.run(lib)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_attention_visible_nan_reaches_its_rows_only(lib):
    """A NaN value among a sequence's keys shows in that sequence and nowhere else; in the prefix, everywhere."""
    for batch in (3, 60):
        b = Batch([20 + i for i in range(batch)], 150, 8, 2, 64, 16, 0, seed=14)
        clean = b.run(lib)[0]
        b.v[int(b.table[1, 0]), 0, 4, 9] = 0x7F
        out = b.run(lib)[0]
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[1, 0:4, 9] = True
        assert torch.equal(torch.isnan(out), hit)
        assert torch.equal(out[~hit], clean[~hit])
        b.v[int(b.prefix_pages[2]), 1, 5, 60] = 0x7F
        hit[:, 4:8, 60] = True
        assert torch.equal(torch.isnan(b.run(lib)[0]), hit)
        b.k[int(b.prefix_pages[1]), 0, 1, 2] = 0xFF
        hit[:, 0:4] = True
        assert torch.equal(torch.isnan(b.run(lib)[0]), hit)


def test_attention_page_out_of_range_is_reported(lib):
    """An index or a length out of range touches nothing out of range and is reported once."""
    for batch in (2, 40):
        b = Batch([100] * batch, 200, 12, 2, 128, 16, 1, seed=15)
        ws = torch.zeros(lib.kv8_prefix_attention_workspace_size(batch, 12, 2, 128, 200, b.table.shape[1], 16),
                         dtype=torch.uint8, device="cuda")
        table, pages, lens = b.table.clone(), b.prefix_pages.clone(), b.lens.clone()
        for what in ("own", "prefix", "long", "negative"):
            b.table, b.prefix_pages, b.lens = table.clone(), pages.clone(), lens.clone()
            if what == "own":
                b.table[1, 2] = b.k.shape[0]
            elif what == "prefix":
                b.prefix_pages[3] = -7
            else:
                b.lens[1] = 10 ** 6 if what == "long" else -1
            b.run(lib, ws=ws)
            assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX, what
            assert lib.w4a8_device_error(ws) == 0
        b.table, b.prefix_pages, b.lens = table, pages, lens
        b.check(*b.run(lib, ws=ws))
        assert lib.w4a8_device_error(ws) == 0


def test_offsets_past_32_bits(lib):
    """A cache of more than 2^31 bytes (and 2^31 codes): the last pages are written, read and attended."""
    h, d, page, pages = 8, 128, 256, 8300   # 2.18e9 codes
    k = torch.zeros(pages, h, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    s = torch.full((h,), 0.05, device="cuda")
    x = _rows(300, h, d, 5).cuda()
    first = (pages - 2) * page
    slots = torch.arange(first, first + 300, dtype=torch.int32, device="cuda")
    lib.kv8_write(x, -x, slots, k, v, s, s)
    got = lib.kv8_read(k, v, s, s, slots)
    small = [torch.zeros(2, h, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    lib.kv8_write(x, -x, slots - first, *small, s, s)
    want = lib.kv8_read(*small, s, s, slots - first)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for batch in (2, 40):
        q = torch.randn(batch, 16, d, device="cuda").to(torch.bfloat16)
        pp = torch.tensor([0], dtype=torch.int32, device="cuda")
        table = torch.tensor([[1]] * batch, dtype=torch.int32, device="cuda")
        lens = torch.tensor([44] * batch, dtype=torch.int32, device="cuda")
        a = lib.kv8_prefix_attention(q, *small, s, s, pp, 256, table, lens, lse=True)
        b = lib.kv8_prefix_attention(q, k, v, s, s, pp + pages - 2, 256, table + pages - 2, lens, lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_another_stream(lib):
    """Allocations inside a call belong to the stream it is given."""
    b = Batch([50] * 8, 300, 16, 2, 128, 32, 1, seed=16)
    want = b.run(lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [b.run(lib, stream=side) for _ in range(20)]
    torch.cuda.current_stream().wait_stream(side)
    for o, z in got:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])


def test_graph_capture_with_growing_lengths(lib):
    """A captured step follows the lengths and pages that stand in device memory at replay."""
    b = Batch([5, 60, 33], 200, 12, 2, 128, 16, 0, seed=17)
    size = lib.kv8_prefix_attention_workspace_size(3, 12, 2, 128, 200, b.table.shape[1], 16)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(b.q), torch.empty(3, 12, device="cuda")
    b.run(lib, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(lib, out=out, lse=lse, ws=ws)
    for lens in ([5, 60, 33], [0, 12, 1], [4, 0, 32]):
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        b.lens_list = lens
        b.check(out, lse)


def test_outputs_and_workspace_stay_in_bounds(lib):
    pad = 4096

    def guarded(nbytes, fill):
        buf = torch.full((2 * pad + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        buf[pad:pad + nbytes] = fill
        return buf, buf[pad:pad + nbytes]

    for lens, prefix, hq, hkv, d, mode in (([3, 0, 40, 17, 90], 130, 48, 8, 128, 0), ([64] * 70, 1100, 12, 2, 64, 1),
                                           ([9], 0, 48, 1, 64, 1), ([5] * 45, 517, 48, 8, 128, 1)):
        b = Batch(lens, prefix, hq, hkv, d, 16, mode, seed=18)
        n = len(lens)
        want = b.run(lib)
        size = lib.kv8_prefix_attention_workspace_size(n, hq, hkv, d, prefix, b.table.shape[1], 16)
        bufs = [guarded(n * hq * d * 2, 0xA5), guarded(n * hq * 4, 0xA5), guarded(size, 0)]
        out = bufs[0][1].view(torch.bfloat16).view(n, hq, d)
        lse = bufs[1][1].view(torch.float32).view(n, hq)
        b.run(lib, out=out, lse=lse, ws=bufs[2][1])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        for buf, _ in bufs:
            assert bool((buf[:pad] == 0xA5).all()) and bool((buf[-pad:] == 0xA5).all())


def test_python_checks_raise_before_a_launch(lib):
    b = Batch([5, 6], 40, 8, 2, 64, 16, 0, seed=19)
    for change in (dict(q=b.q.float()), dict(q=b.q[:, :7]), dict(q=b.q.transpose(0, 1)),
                   dict(out=torch.empty(2, 8, 64, device="cuda")), dict(lse=torch.empty(3, 8, device="cuda"))):
        with pytest.raises((ValueError, lib.W4A8Error)):
            b.run(lib, **change)
    with pytest.raises(lib.W4A8Error):
        b.run(lib, logit_cap=-1.0)
    with pytest.raises(lib.W4A8Error):
        b.run(lib, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for args in ((x, x, slots.long()), (x, x[:, :1], slots), (x, x.half(), slots), (x, x, slots[:1])):
        with pytest.raises(ValueError):
            lib.kv8_write(*args, b.k, b.v, b.ks, b.vs)
    with pytest.raises(ValueError):
        lib.kv8_read(b.k, b.v, b.ks, b.vs[:1], slots)
    with pytest.raises(ValueError):
        lib.kv8_read(b.k, b.v.cpu(), b.ks, b.vs, slots)
