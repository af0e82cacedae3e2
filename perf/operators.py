"""Cases and plain forms of the FP8 key/value cache: writing, reading back, shared-prefix attention.

Every case is one call of one operator, as a decoding or prefilling program makes
it. `run` computes it either through the library (`own`) or in its plain form:
elementary torch operations in 32 bits, rounded once at the end. `exact` gives the
same outputs from the definitions in 64 bits.

The cache is paged, [num_pages, kv heads, page_size, head dim] E4M3 codes, with one
scale per head ("head") or one per token and head ("token").
"""
from types import SimpleNamespace

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def _write(name, tokens, hkv=8, d=128, page=64, scales="head", skip=0, decode=False):
    return {"name": name, "op": "write", "tokens": tokens, "hkv": hkv, "d": d, "page": page, "scales": scales,
            "skip": skip, "decode": decode}


def _read(name, tokens, hkv=8, d=128, page=64, scales="head", skip=0):
    return {"name": name, "op": "read", "tokens": tokens, "hkv": hkv, "d": d, "page": page, "scales": scales,
            "skip": skip}


def _attend(name, batch, prefix, lo, hi, hq=48, hkv=8, d=128, page=64, scales="head", cap=0.0, lse=False):
    return {"name": name, "op": "attend", "batch": batch, "prefix": prefix, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "page": page, "scales": scales, "cap": cap, "lse": lse}


def listed():
    return [
        # One decode step of 32 sequences (Grok-1's 8 key/value heads): the call's latency is what counts.
        _write("write_decode32_head", 32, decode=True),
        # A padded decode batch of 200 slots, of which 37 are padding; small heads and pages.
        _write("write_decode200_d64_token", 200, d=64, page=16, scales="token", skip=37, decode=True),
        # The prompt of the prefill benchmark: 32 sequences of 1024 tokens, scales found as it is written.
        _write("write_prefill32768_token", 32768, scales="token"),
        # Re-reading one prompt of odd length.
        _read("read_1111_head", 1111, page=16),
        # Re-reading the whole prefill batch's cache for a layer that computes in bf16.
        _read("read_32768_token", 32768, scales="token"),
        # One user behind a system prompt: the smallest step, latency.
        _attend("attend_b1_p1024", 1, 1024, 100, 100),
        # The decode benchmark's batch: 32 sequences behind 1024 common tokens, capped logits as Grok-1 has them.
        _attend("attend_b32_p1024_cap", 32, 1024, 1, 256, cap=30.0),
        # Mixtral's heads behind a long system prompt with examples, scales per token.
        _attend("attend_b64_p8192_token", 64, 8192, 1, 512, hq=32, scales="token", lse=True),
        # One shared key/value head, small heads and pages, odd prefix; some sequences have no token of their own yet.
        _attend("attend_b17_p4999_mqa_d64", 17, 4999, 0, 777, hq=16, hkv=1, d=64, page=16, lse=True),
        # Long answers behind a short instruction: the sequences' own tokens are nearly all of the work.
        _attend("attend_b32_p128_long", 32, 128, 4096, 8192, scales="token"),
        # A document of 32768 tokens, 128 questions on it.
        _attend("attend_b128_p32768", 128, 32768, 16, 1024),
        # The largest: 256 samples behind one long context.
        _attend("attend_b256_p65536", 256, 65536, 1, 256, page=128),
    ]


def _spread(rng, lo, hi):
    """A whole number, spread over the logarithm of lo..hi."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return min(hi, max(lo, v))


def draw(rng):
    most = [work(case) for case in listed()]
    while True:  # none that costs more than the largest listed ones
        case = _draw(rng)
        if all(work(case)[n] <= max(w[n] for w in most) for n in ("bytes", "flops")):
            return case


def _draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    scales = rng.choice(["head", "token"])
    if op != "attend":
        tokens = _spread(rng, 1, 32768)
        case = {"op": op, "tokens": tokens, "hkv": rng.choice([1, 2, 5, 8]), "d": d, "page": page, "scales": scales,
                "skip": rng.choice([0, tokens // 7])}
        if op == "write":
            case["decode"] = tokens <= 512 and rng.random() < 0.5
        return case
    hq, hkv = rng.choice([(48, 8), (32, 8), (40, 8), (8, 8), (16, 1), (28, 4)])
    batch = _spread(rng, 1, 256)
    prefix = rng.choice([0, _spread(rng, 1, 65536), _spread(rng, 64, 65536), _spread(rng, 64, 65536)])
    hi = min(8192, 8192 * 32 // batch)
    hi = _spread(rng, 1, hi)
    return {"op": "attend", "batch": batch, "prefix": prefix, "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "scales": scales, "cap": rng.choice([0.0, 0.0, 30.0]),
            "lse": rng.random() < 0.5}


def _lengths(case):
    """The sequences' own lengths, evenly spread over lo..hi (a seed only changes their order)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def work(case):
    hkv, d = case["hkv"], case["d"]
    scale = 8 if case["scales"] == "token" else 0  # bytes of both scales of one token and head
    if case["op"] in ("write", "read"):
        live = case["tokens"] - case["skip"]
        wide, narrow = (live, live) if case["op"] == "write" else (case["tokens"], live)
        n = wide * hkv * d * 4 + narrow * hkv * (2 * d + scale) + 4 * case["tokens"]
        return {"bytes": n + (0 if scale else 8 * hkv), "flops": 4 * live * hkv * d}
    b, p, hq, page = case["batch"], case["prefix"], case["hq"], case["page"]
    lens = _lengths(case)
    keys = p + sum(lens)
    tables = 4 * (-(-p // page) + sum(-(-n // page) for n in lens) + b)
    n = keys * hkv * (2 * d + scale) + (0 if scale else 8 * hkv) + 4 * b * hq * d + (4 * b * hq if case["lse"] else 0)
    return {"bytes": n + tables, "flops": 4 * hq * d * (b * p + sum(lens))}


# ---------------------------------------------------------------- inputs
def _codes(gen, pages, hkv, page, d, scales):
    """A filled cache: E4M3 codes as uint8 and their scales. Keys and values of a model: normal, a few channels of each
    head stronger than the others, tokens of differing strength."""
    x = torch.randn(pages, hkv, page, d, generator=gen, device="cuda")
    x *= 1.0 + 3.0 * (torch.rand(1, hkv, 1, d, generator=gen, device="cuda") > 0.95)
    x *= torch.exp(0.3 * torch.randn(pages, hkv, page, 1, generator=gen, device="cuda"))
    if scales == "token":
        s = x.abs().amax(-1) / torch.tensor(E4M3_MAX, device="cuda")
        x /= s[..., None]
    else:
        s = 0.03 + 0.03 * torch.rand(hkv, generator=gen, device="cuda")
        x /= s[:, None, None]
    return x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), s


def _prepare_rows(case, gen):
    t, hkv, d, page, skip = case["tokens"], case["hkv"], case["d"], case["page"], case["skip"]
    decode = case.get("decode", False)
    pages = t + 3 if decode else -(-t // page) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    if decode:  # every sequence writes into a page of its own
        off = torch.randint(0, page, (t,), generator=gen, device="cuda")
        slots = order[:t] * page + off
    else:
        i = torch.arange(t, device="cuda")
        slots = order[i // page] * page + i % page
    if skip:
        slots[torch.randperm(t, generator=gen, device="cuda")[:skip]] = -1
    # one page more than the cache has: where the plain form puts the tokens that are skipped
    k_all, k_scale = _codes(gen, pages + 1, hkv, page, d, case["scales"])
    v_all, v_scale = _codes(gen, pages + 1, hkv, page, d, case["scales"])
    s = SimpleNamespace(case=case, slots=slots.to(torch.int32), pages=pages, k_all=k_all, v_all=v_all,
                        k_scale_all=k_scale, v_scale_all=v_scale, k_cache=k_all[:pages], v_cache=v_all[:pages])
    token = case["scales"] == "token"
    s.k_scale = k_scale[:pages] if token else k_scale
    s.v_scale = v_scale[:pages] if token else v_scale
    if case["op"] == "write":  # keys and values are columns of the fused projection's output
        qkv = torch.randn(t, 4 * hkv * d, generator=gen, device="cuda").to(torch.bfloat16)
        s.k = qkv[:, 2 * hkv * d:3 * hkv * d].unflatten(1, (hkv, d))
        s.v = qkv[:, 3 * hkv * d:].unflatten(1, (hkv, d))
    else:
        s.k = torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda")
        s.v = torch.empty_like(s.k)
    return s


def _prepare_attend(case, gen):
    b, p, hq, hkv, d, page = (case[n] for n in ("batch", "prefix", "hq", "hkv", "d", "page"))
    lens = torch.tensor(_lengths(case), device="cuda")[torch.randperm(b, generator=gen, device="cuda")]
    most = max(1, -(-case["hi"] // page))
    n_prefix = -(-p // page)
    need = [-(-n // page) for n in _lengths(case)]
    pages = n_prefix + sum(need) + 2
    order = torch.randperm(pages, generator=gen, device="cuda")
    rank = torch.arange(most, device="cuda")[None]
    used = (lens + page - 1) // page
    first = n_prefix + torch.cumsum(used, 0) - used
    table = torch.where(rank < used[:, None], order[(first[:, None] + rank).clamp(max=pages - 1)], -1)
    k_cache, k_scale = _codes(gen, pages, hkv, page, d, case["scales"])
    v_cache, v_scale = _codes(gen, pages, hkv, page, d, case["scales"])
    # what lies behind a sequence's last token in its last page is whatever was there: here codes that are no number
    slot = torch.arange(page, device="cuda")[None]
    last = table.gather(1, (used[:, None] - 1).clamp(min=0))[:, 0]
    last = torch.where(used > 0, last, order[-1])  # the last of the order belongs to nobody
    dead = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    dead[last] = (used > 0)[:, None] & (slot >= (lens - (used - 1) * page)[:, None])
    if p % page:
        dead[order[n_prefix - 1]] = slot[0] >= p % page
    for c in (k_cache, v_cache):
        c.masked_fill_(dead[:, None, :, None], 0x7F)
    qkv = torch.randn(b, (hq + 2 * hkv) * d, generator=gen, device="cuda") * 1.5
    qkv = qkv.to(torch.bfloat16)
    s = SimpleNamespace(case=case, q=qkv[:, :hq * d].unflatten(1, (hq, d)), k_cache=k_cache, v_cache=v_cache,
                        k_scale=k_scale, v_scale=v_scale, prefix_pages=order[:n_prefix].to(torch.int32),
                        page_table=table.to(torch.int32), lens=lens.to(torch.int32), scale=d ** -0.5,
                        out=torch.empty(b, hq, d, dtype=torch.bfloat16, device="cuda"),
                        lse=torch.empty(b, hq, device="cuda") if case["lse"] else None, ws=None)
    if own:  # a decoding program keeps one workspace
        import w4a8_moe_gb300 as lib

        size = lib.kv8_prefix_attention_workspace_size(b, hq, hkv, d, p, most, page)
        s.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_attend if case["op"] == "attend" else _prepare_rows)(case, gen)


# ---------------------------------------------------------------- the framework's calls
def _run_own(s):
    import w4a8_moe_gb300 as lib

    op = s.case["op"]
    if op == "write":
        lib.kv8_write(s.k, s.v, s.slots, s.k_cache, s.v_cache, s.k_scale, s.v_scale)
        return _write_outputs(s)
    if op == "read":
        return list(lib.kv8_read(s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.slots, k_out=s.k, v_out=s.v))
    out, lse = lib.kv8_prefix_attention(s.q, s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.prefix_pages,
                                        s.case["prefix"], s.page_table, s.lens, sm_scale=s.scale,
                                        logit_cap=s.case["cap"], out=s.out, lse=s.lse, ws=s.ws)
    return [out] if lse is None else [out, lse]


def _write_outputs(s):
    out = [s.k_cache.view(torch.float8_e4m3fn), s.v_cache.view(torch.float8_e4m3fn)]
    return out + [s.k_scale, s.v_scale] if s.case["scales"] == "token" else out


# ---------------------------------------------------------------- plain forms
def _plain_write(s):
    page = s.case["page"]
    slots = torch.where(s.slots >= 0, s.slots, s.pages * page).long()
    at, off = slots // page, slots % page
    for x, cache, scale in ((s.k, s.k_all, s.k_scale_all), (s.v, s.v_all, s.v_scale_all)):
        x = x.float()
        if s.case["scales"] == "token":
            size = torch.where(torch.isfinite(x), x, 0.0).abs().amax(-1)
            f = size / torch.full_like(size, E4M3_MAX)
            f = torch.where(f == 0, 1.0, f)
            scale[at, :, off] = f
        else:
            f = scale[None]
        codes = (x / f[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[at, :, off] = codes
    return _write_outputs(s)


def _plain_read(s):
    page = s.case["page"]
    slots = s.slots.clamp(min=0).long()
    at, off = slots // page, slots % page
    outs = []
    for cache, scale in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)):
        x = cache[at, :, off].view(torch.float8_e4m3fn).float()
        f = scale[at, :, off] if s.case["scales"] == "token" else scale[None]
        x = torch.where((s.slots >= 0)[:, None, None], x * f[..., None], 0.0)
        outs.append(x.to(torch.bfloat16))
    return outs


def _plain_keys(s, cache, scale, pages):
    """[..., pages] of a table -> fp32 [kv heads, ..., keys, head dim]."""
    x = cache[pages].view(torch.float8_e4m3fn).float()
    f = scale[pages][..., None] if s.case["scales"] == "token" else scale[:, None, None]
    return (x * f).movedim(-3, 0).flatten(-3, -2)


def _plain_attend(s):
    c = s.case
    b, p, hq, hkv, d, cap = (c[n] for n in ("batch", "prefix", "hq", "hkv", "d", "cap"))
    group = hq // hkv
    q = s.q.float().reshape(b, hkv, group, d).transpose(0, 1)  # [kv heads, batch, group, d]
    table = s.page_table.clamp(min=0).long()
    k_own = _plain_keys(s, s.k_cache, s.k_scale, table)  # [kv heads, batch, keys, d]
    live = torch.arange(k_own.shape[2], device="cuda")[None] < s.lens[:, None]  # [batch, keys]
    s_own = torch.matmul(q, k_own.transpose(-1, -2)) * s.scale
    if cap:
        s_own = cap * torch.tanh(s_own / cap)
    s_own = torch.where(live[None, :, None], s_own, -torch.inf)
    top = s_own.amax(-1, keepdim=True)
    del k_own
    if p:
        pages = s.prefix_pages.long()
        k_all = _plain_keys(s, s.k_cache, s.k_scale, pages)[:, :p]
        s_all = torch.matmul(q.reshape(hkv, b * group, d), k_all.transpose(-1, -2)) * s.scale
        if cap:
            s_all = cap * torch.tanh(s_all / cap)
        s_all = s_all.reshape(hkv, b, group, p)
        top = torch.maximum(top, s_all.amax(-1, keepdim=True))
    top = torch.where(top == -torch.inf, 0.0, top)
    w = torch.exp(s_own - top)
    v_own = torch.where(live[None, :, :, None], _plain_keys(s, s.v_cache, s.v_scale, table), 0.0)
    total, acc = w.sum(-1, keepdim=True), torch.matmul(w, v_own)
    del v_own, s_own, w
    if p:
        w = torch.exp(s_all - top)
        v_all = _plain_keys(s, s.v_cache, s.v_scale, pages)[:, :p]
        total = total + w.sum(-1, keepdim=True)
        acc = acc + torch.matmul(w.reshape(hkv, b * group, p), v_all).reshape(acc.shape)
    out = torch.where(total > 0, acc / torch.where(total > 0, total, 1.0), 0.0)
    out = out.transpose(0, 1).reshape(b, hq, d).to(torch.bfloat16)
    if not c["lse"]:
        return [out]
    lse = (top + torch.log(total))[..., 0].transpose(0, 1).reshape(b, hq)
    return [out, lse]


def run(state):
    if own:
        return _run_own(state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[state.case["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _table64():
    """The value of each of the 256 E4M3 codes, by the format's definition."""
    vals = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v = float("nan") if code & 0x7F == 0x7F else v
        vals.append(-v if code & 0x80 else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _round64(x):
    """x to the nearest E4M3 value, ties to even, saturating."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_write(s):
    page, token = s.case["page"], s.case["scales"] == "token"
    table = _table64()
    keep = torch.nonzero(s.slots >= 0)[:, 0]
    slots = s.slots[keep].long()
    caches, scales = [], []
    for x, cache, scale in ((s.k, s.k_cache, s.k_scale), (s.v, s.v_cache, s.v_scale)):
        vals = table[cache.long()].permute(0, 2, 1, 3).reshape(s.pages * page, s.case["hkv"], s.case["d"])
        x = x[keep].double()
        if token:
            rows = scale.double().permute(0, 2, 1).reshape(s.pages * page, -1)
            f = x.abs().amax(-1) / E4M3_MAX
            f = torch.where(f == 0, torch.ones_like(f), f)
            rows[slots] = f
            scales.append(rows.reshape(s.pages, page, -1).permute(0, 2, 1))
            f = f.float().double()  # codes stand for multiples of the scale as it is kept, in 32 bits
        else:
            f = scale.double().expand(x.shape[0], -1)
        vals[slots] = _round64(x / f[..., None])
        caches.append(vals.reshape(s.pages, page, s.case["hkv"], -1).permute(0, 2, 1, 3))
    return caches + scales


def _exact_read(s):
    page = s.case["page"]
    table = _table64()
    outs = []
    for cache, scale in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)):
        out = torch.zeros(s.case["tokens"], s.case["hkv"], s.case["d"], dtype=torch.float64, device="cuda")
        keep = torch.nonzero(s.slots >= 0)[:, 0]
        slots = s.slots[keep].long()
        rows = table[cache.permute(0, 2, 1, 3).reshape(s.pages * page, s.case["hkv"], -1)[slots].long()]
        f = scale.double()
        f = f.permute(0, 2, 1).reshape(s.pages * page, -1)[slots] if s.case["scales"] == "token" else f[None]
        out[keep] = rows * f[..., None]
        outs.append(out)
    return outs


def _exact_attend(s):
    c = s.case
    b, p, hq, hkv, d, page = (c[n] for n in ("batch", "prefix", "hq", "hkv", "d", "page"))
    table = _table64()

    def gather(cache, scale, pages, n):  # the first n keys of a list of pages, [kv heads, n, d]
        pages = pages[:-(-n // page)].long()
        x = table[cache[pages].long()]
        f = scale.double()
        x = x * (f[pages][..., None] if c["scales"] == "token" else f[:, None, None])
        return x.permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n]

    kp, vp = (gather(x, f, s.prefix_pages, p) for x, f in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)))
    outs = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lses = torch.full((b, hq), -torch.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s.lens.tolist()):
        if p + n == 0:
            continue
        k = torch.cat([kp, gather(s.k_cache, s.k_scale, s.page_table[i], n)], 1)
        v = torch.cat([vp, gather(s.v_cache, s.v_scale, s.page_table[i], n)], 1)
        x = s.q[i].double().reshape(hkv, hq // hkv, d) @ k.transpose(1, 2) * s.scale
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        z = torch.logsumexp(x, -1)
        lses[i] = z.reshape(hq)
        outs[i] = (torch.exp(x - z[..., None]) @ v).reshape(hq, d)
    return [outs, lses] if c["lse"] else [outs]


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)
