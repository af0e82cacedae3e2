"""The key/value cache of 4 bits on the GPU against plain 64-bit forms: writing, reading back, and decode attention."""
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
def bf16(x):
    """fp32 numpy -> the nearest bf16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def quantize(x):
    """[T, H, D] fp32 holding bf16 values -> (codes, steps, least values), by the definition in fp32."""
    x = np.asarray(x, np.float32)
    ok = np.isfinite(x)
    lo = np.where(ok, x, np.float32(np.inf)).min(-1)
    hi = np.where(ok, x, np.float32(-np.inf)).max(-1)
    none = ~ok.any(-1)
    lo, hi = np.where(none, np.float32(0), lo), np.where(none, np.float32(0), hi)
    step = bf16((hi * np.float32(0.5) - lo * np.float32(0.5)) / np.float32(7.5))
    with np.errstate(all="ignore"):
        n = (x * np.float32(0.5) - lo[..., None] * np.float32(0.5)) / (step[..., None] * np.float32(0.5))
    n = np.where(step[..., None] > 0, n, 0)
    nan = np.isnan(x).any(-1)
    codes = np.rint(np.clip(np.where(np.isnan(n), 0, n), 0, 15)).astype(np.uint8)
    codes = np.where(nan[..., None], 0, codes)
    return codes, np.where(nan, np.float32(np.nan), step), np.where(nan, np.float32(np.nan), lo)


def unpack(cache):
    return torch.stack([cache & 15, cache >> 4], -1).flatten(-2)


def rows_of(cache):
    """[pages, H, page, ...] -> [slots, H, ...]"""
    return cache.transpose(1, 2).reshape(cache.shape[0] * cache.shape[2], cache.shape[1], *cache.shape[3:])


def random_cache(gen, pages, h, page, d, spread=0.3, offset=0.5):
    codes = torch.randint(0, 256, (pages, h, page, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
    size = torch.exp(spread * torch.randn(pages, h, page, generator=gen, device="cuda"))
    step = 0.3 * size
    least = (-2.2 + offset * torch.randn(pages, h, page, generator=gen, device="cuda")) * size
    return codes, torch.stack([step, least], -1).to(torch.bfloat16)


# ---------------------------------------------------------------- write and read
def _rows(t, h, d, seed, special=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=gen) * torch.exp(torch.randn(t, h, 1, generator=gen))
    x += torch.randn(t, h, 1, generator=gen)
    if special:
        x[0, 0, :] = 0
        x[1, 0, :] = 1.625
        x[2, 0, :] = float("inf")
        x[t // 2, 0, 3] = float("inf")
        x[t // 2, 0, 5] = float("-inf")
        x[t // 3, h - 1, d - 1] = float("nan")
        x[t - 1, 0, :] = torch.linspace(-3.2e38, 3.2e38, d, dtype=torch.float64)
        x[t - 2, 0, :] = torch.linspace(1e-40, 3e-39, d, dtype=torch.float64)
        x[t - 3, 0, :] = torch.linspace(2.0 ** -70, 2.0 ** -66, d)
        x[t - 4, 0, :] = 100 + torch.arange(d) % 3
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("t,h,d,page,fused,skip", [
    (1, 8, 128, 64, False, 0), (1, 1, 64, 16, True, 0), (10, 5, 128, 16, True, 2), (33, 3, 64, 32, False, 1),
    (257, 6, 128, 128, True, 40), (1000, 1, 64, 256, False, 7), (4099, 2, 128, 64, False, 0), (9, 2, 64, 32, True, 9),
])
def test_write(lib, t, h, d, page, fused, skip):
    """Codes, steps and least values are those of the definition; other slots keep what they held."""
    pages = -(-t // page) + 2
    gen = torch.Generator(device="cuda").manual_seed(t)
    caches = [random_cache(gen, pages, h, page, d) for _ in range(2)]
    before = [(rows_of(unpack(c)).cpu().numpy().copy(), rows_of(s).float().cpu().numpy().copy()) for c, s in caches]
    slots = np.random.default_rng(t).permutation(pages * page)[:t].astype(np.int32)
    for i, bad in zip(range(0, t, max(1, t // max(skip, 1))) if skip else (), [-1, pages * page, 2 ** 31 - 1, -2 ** 31] * t):
        slots[i] = bad
    k, v = _rows(t, h, d, t + 1, special=t > 8), _rows(t, h, d, t + 2)
    if fused:
        qkv = torch.zeros(t, 3 * h * d + 8, dtype=torch.bfloat16)
        qkv[:, 8 + h * d:8 + 2 * h * d] = k.reshape(t, -1)
        qkv[:, 8 + 2 * h * d:] = v.reshape(t, -1)
        qkv = qkv.cuda()
        kg = qkv[:, 8 + h * d:8 + 2 * h * d].unflatten(1, (h, d))
        vg = qkv[:, 8 + 2 * h * d:].unflatten(1, (h, d))
    else:
        kg, vg = k.cuda(), v.cuda()
    (kc, ks), (vc, vs) = caches
    lib.kv4_write(kg, vg, torch.from_numpy(slots).cuda(), kc, vc, ks, vs)
    ok = (slots >= 0) & (slots < pages * page)
    for x, (cache, scale), (codes, pair) in ((k, caches[0], before[0]), (v, caches[1], before[1])):
        c, s, m = quantize(x.float().numpy())
        codes[slots[ok]] = c[ok]
        pair[slots[ok]] = np.stack([s, m], -1)[ok]
        assert np.array_equal(rows_of(unpack(cache)).cpu().numpy(), codes)
        assert np.array_equal(rows_of(scale).float().cpu().numpy(), pair, equal_nan=True)


@pytest.mark.parametrize("lo,hi", [(-1.0, 1.0), (0.0, 15.0), (-0.3, 2.9), (-448.0, 0.01), (-1e-30, 1e-30), (1e30, 3e30),
                                   (-3e38, 3e38), (0.0, 1e-37), (5.0, 5.5), (-2.0 ** -61, 2.0 ** -59)])
def test_write_code_of_every_bf16_value(lib, lo, hi):
    """Codes are those of the fp32 quotient for every bf16 value between a row's least and largest."""
    bits = np.arange(0x10000, dtype=np.uint32) << 16
    vals = bits.view(np.float32)
    vals = vals[np.isfinite(vals)]
    lo, hi = bf16([lo, hi])
    vals = vals[(vals >= lo) & (vals <= hi)]
    vals = np.random.default_rng(0).permutation(vals)
    per = 62
    vals = np.concatenate([vals, np.full(-len(vals) % per, lo, np.float32)]).reshape(-1, 1, per)
    t = vals.shape[0]
    x = np.concatenate([vals, np.full((t, 1, 1), lo, np.float32), np.full((t, 1, 1), hi, np.float32)], -1)
    xg = torch.from_numpy(x).to(torch.bfloat16).cuda()
    pages = -(-t // 256)
    kc, vc = (torch.zeros(pages, 1, 256, 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, 1, 256, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.kv4_write(xg, xg, torch.arange(t, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    want, step, least = quantize(x)
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(rows_of(unpack(c)).cpu().numpy()[:t], want)
        assert np.array_equal(rows_of(s).float().cpu().numpy()[:t], np.stack([step, least], -1))


@pytest.mark.parametrize("t,h,d,page", [(1, 1, 64, 16), (19, 5, 128, 32), (333, 8, 64, 64), (2049, 2, 128, 256)])
def test_read(lib, t, h, d, page):
    gen = torch.Generator(device="cuda").manual_seed(t)
    pages = 5 + t // page
    (kc, ks), (vc, vs) = (random_cache(gen, pages, h, page, d) for _ in range(2))
    ks[0, 0, 4] = float("nan")
    slots = np.random.default_rng(t).integers(0, pages * page, t).astype(np.int32)          # may repeat
    slots[0] = 4
    for i, bad in zip(range(1, t, 7), [-1, pages * page, -2 ** 31] * t):
        slots[i] = bad
    wide = torch.full((t, 3, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = lib.kv4_read(kc, vc, ks, vs, torch.from_numpy(slots).cuda(), k_out=wide[:, 0], v_out=wide[:, 2])
    assert bool((wide[:, 1] == 7.0).all())
    ok = (slots >= 0) & (slots < pages * page)
    for got, cache, scale in ((k, kc, ks), (v, vc, vs)):
        c, s = rows_of(unpack(cache)).cpu().numpy(), rows_of(scale).float().cpu().numpy().astype(np.float64)
        want = np.zeros((t, h, d), np.float32)
        want[ok] = (c * s[..., :1] + s[..., 1:])[slots[ok]]   # exact in 64 bits; fp32, then bf16
        assert np.array_equal(got.float().cpu().numpy(), bf16(want), equal_nan=True)
        assert np.all(got.float().cpu().numpy()[~ok] == 0)


def test_write_then_read_is_within_half_a_step(lib):
    t, h, d, page = 100, 4, 128, 16
    x = _rows(t, h, d, 3).cuda()
    cache = [torch.zeros(8, h, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(8, h, page, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.arange(t, dtype=torch.int32, device="cuda") + 5
    lib.kv4_write(x, x, slots, *cache, *scales)
    k, v = lib.kv4_read(*cache, *scales, slots)
    assert torch.equal(k, v)
    x = x.float()
    step = (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15
    # half a step, 2^-8 off at most, the largest value 15 times that beyond the last code; and the reading's bf16
    bound = step * (0.5 + 16 * 2.0 ** -8) + x.abs().amax(-1, keepdim=True) * 2.0 ** -8
    assert bool(((k.float() - x).abs() <= bound * 1.01).all())


# ---------------------------------------------------------------- attention
class Batch:
    """A paged 4-bit cache and query tokens: `drafts` of each sequence, the last of which sees all of its keys."""

    def __init__(self, lens, hq, hkv, d, page, cap=0.0, seed=0, q_scale=1.5, spread=0.3, offset=0.5, extra=1, drafts=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.d, self.page, self.cap, self.scale = hq, hkv, d, page, cap, d ** -0.5
        need = [-(-n // page) for n in lens]
        most = max(need + [1]) + extra
        pages = sum(need) + 1
        order = torch.randperm(pages, generator=gen, device="cuda").tolist()
        table = np.full((len(lens), most), -1, np.int32)
        self.k, self.ks = random_cache(gen, pages, hkv, page, d, spread, offset)
        self.v, self.vs = random_cache(gen, pages, hkv, page, d, spread, offset)
        at = 0
        for i, n in enumerate(lens):
            table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            if n % page:   # what lies behind the last token is no number
                pg = int(table[i, need[i] - 1])
                self.ks[pg, :, n % page:] = float("nan")
                self.vs[pg, :, n % page:] = float("inf")
        self.table = torch.from_numpy(table).cuda()
        self.seqs_list = [i for i in range(len(lens)) for _ in range(drafts)]
        self.lens_list = [max(n - drafts + 1 + j, 0) for n in lens for j in range(drafts)]
        self.seqs = torch.tensor(self.seqs_list, dtype=torch.int32, device="cuda") if drafts > 1 else None
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32, device="cuda")
        t = len(self.lens_list)
        self.q = (torch.randn(t, hq, d, generator=gen, device="cuda") * q_scale).to(torch.bfloat16)

    def run(self, lib, **kw):
        args = dict(seqs=self.seqs, sm_scale=self.scale, logit_cap=self.cap, lse=True)
        args.update(kw)
        q = args.pop("q", self.q)
        return lib.kv4_attention(q, self.k, self.v, self.ks, self.vs, self.table, self.lens, **args)

    def keys(self, t):
        """fp64 codes [heads, keys, D], steps and least values [heads, keys, 1] of K and V, as one token sees them."""
        n = self.lens_list[t]
        pg = self.table[self.seqs_list[t]][:-(-n // self.page)].long()
        out = []
        for cache, s in ((self.k, self.ks), (self.v, self.vs)):
            c = unpack(cache[pg]).double().transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :n]
            f = s[pg].double().transpose(0, 1).reshape(self.hkv, -1, 2)[:, :n]
            out += [c, f[..., :1], f[..., 1:]]
        return out

    def check(self, got, lse, every=1):
        """Elementwise bounds from the arithmetic, none fitted to the outcome. The value that the kernel rounds to bf16
        lies within `tol` of the exact one; rounding is monotone, so the output lies between the roundings of the
        interval's ends. A score's error: fp32 sums of D products and of D queries (2^-23 per addition of the sum of
        magnitudes, of steps times codes and of least values apart), q's elements in f16 below its row's largest (2^-35
        of it each), the scaling and exponent (2^-21 of the score's size plus 2^-21), the cap's tanh (2^-20 of the cap).
        A weight's f16 rounding: 2^-11 of it, plus the tail of f16's range: 2^-32 of the largest product of a weight with
        its value's size, for each key, times a code."""
        assert bool(torch.isfinite(got.float()).all())
        group = self.hq // self.hkv
        for t in range(0, len(self.lens_list), every):
            n = self.lens_list[t]
            o, z = got[t].double(), lse[t].double()
            if n == 0:
                assert bool((o == 0).all()) and bool((z == -torch.inf).all())
                continue
            kc, kst, kl, vc, vst, vl = self.keys(t)
            q = self.q[t].double().reshape(self.hkv, group, self.d)
            s = q @ (kc * kst + kl).transpose(1, 2) * self.scale
            size = (q.abs() @ (kc * kst.abs() + kl.abs()).transpose(1, 2)) * abs(self.scale)
            tiny = q.abs().amax(-1, keepdim=True) * (kc * kst.abs()).sum(-1)[:, None] * abs(self.scale)
            ds = size * (self.d + 8) * 2.0 ** -23 + tiny * 2.0 ** -35 + 2.0 ** -21 * s.abs()
            if self.cap:
                s = self.cap * torch.tanh(s / self.cap)
                ds = ds + 2.0 ** -20 * self.cap
            ds = ds.amax(-1, keepdim=True) + 2.0 ** -21
            w = torch.softmax(s, -1)
            want = w @ (vc * vst + vl)
            mag = w @ (vc * vst.abs() + vl.abs())
            top = (w * torch.maximum(vst.abs(), vl.abs())[..., 0][:, None]).amax(-1, keepdim=True)
            floor = top * 2.0 ** -32 * vc.sum(1)[:, None]
            tol = (2.0 ** -11 + 2 * ds) * mag * 1.01 + floor + 1e-30
            o = o.reshape(want.shape)
            low, high = (x.float().to(torch.bfloat16).double() for x in (want - tol, want + tol))
            assert bool(((o >= low) & (o <= high)).all()), (t, float(((o - want).abs() / tol).max()))
            zw = torch.logsumexp(s, -1)
            zerr = (z.reshape(zw.shape) - zw).abs()
            ztol = ds[..., 0] + 2.0 ** -21 * (1 + zw.abs())
            assert bool((zerr <= ztol).all()), (t, float((zerr / ztol).max()))


@pytest.mark.parametrize("hq,hkv,d,page", [
    (48, 8, 128, 64), (32, 8, 128, 16), (8, 8, 64, 32), (16, 1, 64, 16), (9, 1, 128, 128), (48, 1, 128, 256),
    (28, 4, 64, 64), (34, 2, 64, 16), (16, 1, 128, 16), (1, 1, 128, 32),
])
def test_attention_heads_and_pages(lib, hq, hkv, d, page):
    """Every head layout and page size; lengths of zero, one, around a half unit, a unit and a page."""
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 48, 49, page - 1, page, page + 1, 200, 3]
    b = Batch(lens, hq, hkv, d, page, seed=hq)
    b.check(*b.run(lib))


@pytest.mark.parametrize("hq,hkv,d,page,drafts", [(48, 8, 128, 64, 4), (16, 1, 64, 16, 2), (32, 8, 128, 32, 7)])
def test_attention_several_tokens_of_a_sequence(lib, hq, hkv, d, page, drafts):
    """Drafted tokens: each sees the keys before it and its own; sequences shorter than their drafts leave some without."""
    b = Batch([0, 3, drafts, 16, 17, 40, 65, 300, 2], hq, hkv, d, page, seed=drafts, drafts=drafts)
    b.check(*b.run(lib))
    # tokens in any order, sequences left out, padding behind (whose sequence is not read)
    perm = torch.randperm(len(b.seqs_list), generator=torch.Generator().manual_seed(1)).tolist()[:-3]
    b.q = torch.cat([b.q[perm], b.q[:2]])
    b.seqs = torch.cat([b.seqs[perm], torch.tensor([-1, 10 ** 9], dtype=torch.int32, device="cuda")])
    b.lens = torch.cat([b.lens[perm], torch.zeros(2, dtype=torch.int32, device="cuda")])
    ws = torch.zeros(lib.kv4_attention_workspace_size(len(perm) + 2, hq, hkv, d, b.table.shape[1], page),
                     dtype=torch.uint8, device="cuda")
    b.seqs_list = [b.seqs_list[i] for i in perm] + [0, 0]
    b.lens_list = [b.lens_list[i] for i in perm] + [0, 0]
    out, lse = b.run(lib, ws=ws)
    b.check(out, lse)
    assert lib.w4a8_device_error(ws) == 0
    empty = [i for i, n in enumerate(b.lens_list) if n == 0]
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -torch.inf).all())


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 8, 64, 32), (12, 4, 128, 16), (32, 8, 128, 64), (16, 4, 64, 16), (40, 8, 64, 16),
                                           (14, 2, 128, 32), (8, 1, 128, 16), (18, 2, 64, 64)])
def test_attention_runs_of_tokens(lib, hq, hkv, d, page):
    """Runs of neighbours of one sequence, of every length: shorter and longer than what a tile of rows holds, the same
    sequence in several runs, lengths in any order within a run, tokens without keys inside one; few and many sequences."""
    for rows, seed, runs in ((6, 0, (1, 2, 3, 5, 8, 16, 17, 33, 1, 2, 4)), (60, 1, (1, 2, 3, 5, 8, 16, 17, 33, 1, 2, 4)),
                             (40, 2, (100, 61, 200, 1, 7, 140, 3))):   # (across 128 tokens, which a block sums at once)
        b = Batch([(53 * i) % 400 + 20 for i in range(rows)], hq, hkv, d, page, seed=seed + hq)
        full = b.lens_list
        rng = np.random.default_rng(seed)
        seqs, lens = [], []
        for run in runs:
            i = int(rng.integers(0, min(rows, 6)))
            seqs += [i] * run
            some = full[i] - np.arange(run)[::-1] if run % 2 else rng.integers(0, full[i] + 1, run)
            lens += [max(int(n), 0) for n in some]
        b.seqs_list, b.lens_list = seqs, lens
        b.seqs = torch.tensor(seqs, dtype=torch.int32, device="cuda")
        b.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(seed)
        b.q = (torch.randn(len(seqs), hq, d, generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
        b.check(*b.run(lib), every=1 if len(seqs) < 100 else 5)


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (6, 1, 128), (8, 2, 128)])
def test_attention_a_token_does_not_see_what_is_behind_it(lib, hq, hkv, d):
    """Keys and values that are no numbers, behind a token's last key but before its neighbour's, leave it as it was."""
    b = Batch([100, 70, 33], hq, hkv, d, 16, seed=41, drafts=4)
    clean = b.run(lib)
    for which in ("ks", "vs"):
        for bad in (float("nan"), float("inf")):
            keep = getattr(b, which).clone()
            for i, n in enumerate((100, 70, 33)):   # the last draft's own key
                getattr(b, which)[int(b.table[i, (n - 1) // 16]), :, (n - 1) % 16] = bad
            out, lse = b.run(lib)
            last = torch.arange(12) % 4 == 3
            assert torch.equal(out[~last], clean[0][~last]) and torch.equal(lse[~last], clean[1][~last])
            if bad != bad:   # (a score of minus infinity is a weight of zero)
                assert bool(torch.isnan(out[last]).any(-1).all())
            getattr(b, which).copy_(keep)


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (3, 1, 128)])
def test_attention_largest_batch(lib, hq, hkv, d):
    """4096 tokens, the most a call takes (every 37th checked)."""
    b = Batch([(i * 7) % 70 for i in range(4096)], hq, hkv, d, 16, seed=20)
    b.check(*b.run(lib), every=37)
    b = Batch([(i * 7) % 70 for i in range(1024)], hq, hkv, d, 16, seed=20, drafts=4)
    b.check(*b.run(lib), every=37)


def test_attention_shared_memory_at_its_default_limit(lib):
    """Batches whose prefix sums take a block's shared memory past the 48 KB that need no asking for."""
    for batch in range(1524, 1540):
        b = Batch([i % 5 for i in range(batch)], 1, 1, 128, 16, seed=batch)
        b.check(*b.run(lib), every=211)


@pytest.mark.parametrize("batch,hq,hkv,d,own,extra,page", [
    (1, 16, 1, 128, 9000, 1, 64),     # many pieces a row, joined by eight warps
    (3, 8, 8, 64, 5000, 1, 16),
    (70, 8, 1, 64, 1500, 1, 64),      # joined by four
    (70, 12, 1, 64, 2000, 200, 32),
    (30, 28, 4, 128, 1000, 1, 16),    # by two
    (70, 16, 1, 128, 900, 200, 64),
    (260, 6, 2, 128, 70, 1, 64),      # four units a warp
    (5, 128, 16, 128, 3000, 5000, 128),   # tables far wider than the lengths
])
def test_attention_long_contexts(lib, batch, hq, hkv, d, own, extra, page):
    """Every way of cutting the keys into pieces and of joining them."""
    lens = [own - 37 * i % own if i % 6 != 5 else i % 3 for i in range(batch)]
    b = Batch(lens, hq, hkv, d, page, seed=own, extra=extra)
    b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [2, 40])
def test_attention_logit_cap(lib, batch):
    """Capped scores, from far below the cap to far above it."""
    for q_scale in (0.1, 1.5, 30.0):
        b = Batch([500 + i for i in range(batch)], 48, 8, 128, 64, cap=30.0, seed=4, q_scale=q_scale)
        b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [1, 64])
def test_attention_peaked_and_flat(lib, batch):
    """Scores spread over hundreds (one key wins) and all equal (the mean of the values)."""
    for q_scale in (40.0, 0.0):
        b = Batch([1000] * batch, 16, 2, 128, 32, seed=8, q_scale=q_scale)
        b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [1, 64])
def test_attention_scales_far_apart(lib, batch):
    """Steps over many binades, rising along the keys and tiny throughout; least values far larger than the steps;
    steps of zero (rows of one value) and rows of zeros."""
    b = Batch([1000] * batch, 16, 2, 128, 32, seed=9, spread=1.5, q_scale=0.3)
    b.check(*b.run(lib))
    b.vs *= 2.0 ** -60
    b.ks *= 2.0 ** 20
    b.scale *= 2.0 ** -20
    b.check(*b.run(lib))
    b = Batch([1000] * batch, 16, 2, 128, 32, seed=10, q_scale=0.3)
    b.vs[..., 1] += 300.0
    b.check(*b.run(lib))
    b.vs[::2, ..., 0] = 0
    b.check(*b.run(lib))
    b.vs[::3] = 0
    b.ks[1::3, ..., 0] = 0
    b.check(*b.run(lib))


@pytest.mark.parametrize("batch", [2, 50])
def test_attention_small_and_large_queries(lib, batch):
    """q outside f16's range, with sm_scale taking it back; a negative sm_scale."""
    for mul in (2.0 ** 100, 2.0 ** -100):
        b = Batch([240] * batch, 12, 2, 128, 32, seed=10)
        b.q = (b.q.double() * mul).to(torch.bfloat16)
        b.scale /= mul
        b.check(*b.run(lib))
    b = Batch([240] * batch, 12, 2, 128, 32, seed=10)
    b.scale = -b.scale
    b.check(*b.run(lib))


def test_attention_negative_steps(lib):
    """A cache written by another program may count its codes from above."""
    b = Batch([240] * 3, 12, 2, 128, 32, seed=30)
    b.ks[::2, ..., 0] *= -1
    b.vs[1::2, ..., 0] *= -1
    b.check(*b.run(lib))


def test_attention_strided_queries_and_tables(lib):
    """q as columns of a fused projection, the page table as columns of a larger one."""
    b = Batch([130, 0, 170, 9], 12, 2, 64, 16, seed=11)
    want = b.run(lib)
    qkv = torch.randn(4, 12 * 64 + 256, device="cuda").to(torch.bfloat16)
    qkv[:, 128:128 + 12 * 64] = b.q.reshape(4, -1)
    big = torch.full((4, b.table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    big[:, 3:3 + b.table.shape[1]] = b.table
    b.table = big[:, 3:3 + b.table.shape[1]]
    got = b.run(lib, q=qkv[:, 128:128 + 12 * 64].unflatten(1, (12, 64)))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("batch,own", [(3, 500), (60, 700), (1, 20000)])
def test_attention_same_bits_each_call_and_any_workspace_contents(lib, batch, own):
    b = Batch([own - i for i in range(batch)], 48, 8, 128, 64, seed=12)
    size = lib.kv4_attention_workspace_size(batch, 48, 8, 128, b.table.shape[1], 64)
    first = b.run(lib)
    for fill in (0x00, 0x7F, 0xFF):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        got = b.run(lib, ws=ws)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
        assert lib.w4a8_device_error(ws) == 0
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        got = b.run(lib)
        differ += (got[0] != first[0]).sum() + (got[1] != first[1]).sum()
    assert int(differ) == 0


def test_attention_without_lse_and_without_keys(lib):
    b = Batch([0, 0, 0], 8, 2, 64, 16, seed=13)
    out, lse = b.run(lib)
    b.check(out, lse)
    only, none = b.run(lib, lse=None)
    assert none is None and torch.equal(only, out)
    b.table = b.table[:, :0]
    got = b.run(lib)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_attention_visible_nan_reaches_its_rows_only(lib):
    """A row that is no number among a sequence's keys shows in that sequence's heads and nowhere else."""
    for batch in (3, 60):
        for which in ("vs", "ks"):
            b = Batch([150 + i for i in range(batch)], 8, 2, 64, 16, seed=14)
            clean = b.run(lib)[0]
            getattr(b, which)[int(b.table[1, 0]), 0, 4] = float("nan")
            out = b.run(lib)[0]
            hit = torch.zeros_like(out, dtype=torch.bool)
            hit[1, 0:4] = True
            assert torch.equal(torch.isnan(out), hit)
            assert torch.equal(out[~hit], clean[~hit])


def test_attention_index_out_of_range_is_reported(lib):
    """A page, a length or a sequence out of range touches nothing out of range and is reported once."""
    for batch in (2, 40):
        b = Batch([300] * batch, 12, 2, 128, 16, seed=15, drafts=2)
        t = 2 * batch
        ws = torch.zeros(lib.kv4_attention_workspace_size(t, 12, 2, 128, b.table.shape[1], 16), dtype=torch.uint8,
                         device="cuda")
        table, lens, seqs = b.table.clone(), b.lens.clone(), b.seqs.clone()
        for what in ("page", "odd page", "long", "negative", "seq"):
            b.table, b.lens, b.seqs = table.clone(), lens.clone(), seqs.clone()
            if what == "page":
                b.table[1, 2] = b.k.shape[0]
            elif what == "odd page":
                b.table[1, 3] = -7
            elif what == "seq":
                b.seqs[1] = batch
            else:
                b.lens[1] = 10 ** 6 if what == "long" else -1
            b.run(lib, ws=ws)
            assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX, what
            assert lib.w4a8_device_error(ws) == 0
        b.table, b.lens, b.seqs = table, lens, seqs
        b.check(*b.run(lib, ws=ws))
        assert lib.w4a8_device_error(ws) == 0


def test_offsets_past_32_bits(lib):
    """A cache of more than 2^31 bytes: the last pages are written, read and attended."""
    h, d, page, pages = 8, 128, 256, 16500   # 2.16e9 bytes of codes
    k = torch.zeros(pages, h, page, d // 2, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.zeros(pages, h, page, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _rows(300, h, d, 5).cuda()
    first = (pages - 2) * page
    slots = torch.arange(first, first + 300, dtype=torch.int32, device="cuda")
    lib.kv4_write(x, -x, slots, k, v, ks, vs)
    got = lib.kv4_read(k, v, ks, vs, slots)
    small = [torch.zeros(2, h, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(2, h, page, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lib.kv4_write(x, -x, slots - first, *small, *scales)
    want = lib.kv4_read(*small, *scales, slots - first)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q = torch.randn(2, 16, d, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[0, 1]] * 2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([300, 257], dtype=torch.int32, device="cuda")
    a = lib.kv4_attention(q, *small, *scales, table, lens, lse=True)
    b = lib.kv4_attention(q, k, v, ks, vs, table + pages - 2, lens, lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_another_stream(lib):
    """Allocations inside a call belong to the stream it is given."""
    b = Batch([350] * 8, 16, 2, 128, 32, seed=16)
    want = b.run(lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [b.run(lib, stream=side) for _ in range(20)]
    torch.cuda.current_stream().wait_stream(side)
    for o, z in got:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])


def test_two_calls_at_once(lib):
    """Two calls on two streams, each with its workspace, large and small: each gives the bits it gives alone."""
    a, b = Batch([6000] * 40, 32, 8, 128, 64, seed=61), Batch([200, 7000, 3], 8, 2, 64, 16, seed=62, drafts=2)
    ws = [torch.zeros(lib.kv4_attention_workspace_size(n, hq, hkv, d, 1, 16), dtype=torch.uint8, device="cuda")
          for n, hq, hkv, d in ((40, 32, 8, 128), (6, 8, 2, 64))]
    want = [x.run(lib, ws=w) for x, w in zip((a, b), ws)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    differ = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(40):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got = x.run(lib, ws=ws[i])
                differ[i] += (got[0] != want[i][0]).sum() + (got[1] != want[i][1]).sum()
    torch.cuda.synchronize()
    assert [int(x) for x in differ] == [0, 0] and all(lib.w4a8_device_error(w) == 0 for w in ws)


def test_graph_capture_with_growing_lengths(lib):
    """A captured step (write, attention, reading back) follows the lengths and pages that stand in device memory."""
    b = Batch([5, 60, 33], 12, 2, 128, 16, seed=17)
    ws = torch.zeros(lib.kv4_attention_workspace_size(3, 12, 2, 128, b.table.shape[1], 16), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(b.q), torch.empty(3, 12, device="cuda")
    x = _rows(3, 2, 128, 4).cuda()
    slots = torch.tensor([int(b.table[0, 0]) * 16 + 1, -1, int(b.table[2, 0]) * 16], dtype=torch.int32, device="cuda")
    back = [torch.empty_like(x) for _ in range(2)]

    def step():
        lib.kv4_write(x, x, slots, b.k, b.v, b.ks, b.vs)
        b.run(lib, out=out, lse=lse, ws=ws)
        lib.kv4_read(b.k, b.v, b.ks, b.vs, slots, k_out=back[0], v_out=back[1])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, lens in enumerate(([5, 60, 33], [0, 12, 1], [4, 0, 32])):
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        x.copy_(_rows(3, 2, 128, 40 + i))
        graph.replay()
        b.lens_list = lens
        b.check(out, lse)
        assert torch.equal(back[0], back[1]) and bool((back[0][1] == 0).all())


def test_outputs_and_workspace_stay_in_bounds(lib):
    pad = 4096

    def guarded(nbytes, fill):
        buf = torch.full((2 * pad + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        buf[pad:pad + nbytes] = fill
        return buf, buf[pad:pad + nbytes]

    for lens, hq, hkv, d in (([3, 0, 40, 17, 900], 48, 8, 128), ([64] * 70, 12, 2, 64), ([9], 40, 1, 64), ([77] * 45, 48, 8, 128)):
        b = Batch(lens, hq, hkv, d, 16, seed=18)
        n = len(lens)
        want = b.run(lib)
        size = lib.kv4_attention_workspace_size(n, hq, hkv, d, b.table.shape[1], 16)
        bufs = [guarded(n * hq * d * 2, 0xA5), guarded(n * hq * 4, 0xA5), guarded(size, 0)]
        out = bufs[0][1].view(torch.bfloat16).view(n, hq, d)
        lse = bufs[1][1].view(torch.float32).view(n, hq)
        b.run(lib, out=out, lse=lse, ws=bufs[2][1])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        for buf, _ in bufs:
            assert bool((buf[:pad] == 0xA5).all()) and bool((buf[-pad:] == 0xA5).all())


def test_python_checks_raise_before_a_launch(lib):
    b = Batch([5, 6], 8, 2, 64, 16, seed=19)
    for change in (dict(q=b.q.float()), dict(q=b.q[:, :7]), dict(q=b.q.transpose(0, 1)),
                   dict(out=torch.empty(2, 8, 64, device="cuda")), dict(lse=torch.empty(3, 8, device="cuda")),
                   dict(seqs=torch.zeros(2, dtype=torch.int64, device="cuda")),
                   dict(seqs=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(logit_cap=-1.0),
                   dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, lib.W4A8Error)):
            b.run(lib, **change)
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for args in ((x, x, slots.long()), (x, x[:, :1], slots), (x, x.half(), slots), (x, x, slots[:1])):
        with pytest.raises(ValueError):
            lib.kv4_write(*args, b.k, b.v, b.ks, b.vs)
    for scale in (b.vs.float(), b.vs[:1], b.vs[..., 0]):
        with pytest.raises(ValueError):
            lib.kv4_read(b.k, b.v, b.ks, scale, slots)
    with pytest.raises(ValueError):
        lib.kv4_read(b.k, b.v.cpu(), b.ks, b.vs, slots)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (40, 8, 64)])
def test_attention_very_many_units(lib, hq, hkv, d):
    """So many keys that the shares go by the blocks' places: right, the same bits every time, the workspace's counters
    left at zero, and larger and smaller calls in turn on one workspace."""
    b = Batch([5000 + 331 * i % 3000 for i in range(40)], hq, hkv, d, 64, seed=50)
    few = Batch([300, 20, 7], hq, hkv, d, 64, seed=51)
    ws = torch.zeros(lib.kv4_attention_workspace_size(40, hq, hkv, d, 1, 64), dtype=torch.uint8, device="cuda")
    first, small = b.run(lib, ws=ws), few.run(lib, ws=ws)
    b.check(*first, every=7)
    few.check(*small)
    assert bool((ws[:256] == 0).all())
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        for x, want in ((b, first), (few, small)):
            got = x.run(lib, ws=ws)
            differ += (got[0] != want[0]).sum() + (got[1] != want[1]).sum()
    assert int(differ) == 0 and lib.w4a8_device_error(ws) == 0
    # beside other work on the GPU: blocks come to other places
    side = torch.cuda.Stream()
    m = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            m = torch.relu(m) + 0.5
        got = b.run(lib, ws=ws)
        differ += (got[0] != first[0]).sum() + (got[1] != first[1]).sum()
    torch.cuda.synchronize()
    assert int(differ) == 0 and lib.w4a8_device_error(ws) == 0 and bool((ws[:256] == 0).all())


def test_attention_header_that_is_not_zero_is_reported(lib):
    """Counters that a call did not leave behind: the call ends, and says so."""
    b = Batch([7000] * 40, 32, 8, 128, 64, seed=52)
    ws = torch.zeros(lib.kv4_attention_workspace_size(40, 32, 8, 128, 1, 64), dtype=torch.uint8, device="cuda")
    want = b.run(lib, ws=ws)
    ws[64:80] = 0x7F
    b.run(lib, ws=ws)
    assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX
    got = b.run(lib, ws=ws)   # the call has put them right
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and lib.w4a8_device_error(ws) == 0
