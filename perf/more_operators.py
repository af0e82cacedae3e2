"""Cases and plain forms of what stands around the paged key/value cache in a serving step: page tables and slots from
request lengths, the norm and rotation of queries and keys (alone, or straight into the FP8 cache), and a cache of 4 bits
with its decode attention.

Every case is one pass of one operator, as a decoding or prefilling program makes it. `run` computes it either through the
library (`own`) or in its plain form: elementary torch operations in 32 bits (64 for angles), rounded once at the end.
`exact` gives the same outputs from the definitions in 64 bits.
"""
import math
from types import SimpleNamespace

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def _rope(name, tokens, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, scaling="none", far=8192, decode=False):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "inter": inter,
            "norm": norm, "scaling": scaling, "far": far, "decode": decode}


def _write(name, tokens, hq=48, hkv=8, d=128, rot=128, inter=False, norm=True, scaling="none", far=8192, decode=False,
           page=64, scales="token", skip=0):
    return {"name": name, "op": "rope_write", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "inter": inter,
            "norm": norm, "scaling": scaling, "far": far, "decode": decode, "page": page, "scales": scales, "skip": skip}


def _pages(name, batch, ctx, new_lo, new_hi, page=64, pad=0, short=False):
    return {"name": name, "op": "pages", "batch": batch, "ctx": ctx, "new_lo": new_lo, "new_hi": new_hi, "page": page,
            "pad": pad, "short": short}


def _rows4(name, tokens, hkv=8, d=128, page=64, skip=0, decode=False):
    return {"name": name, "op": "rows4", "tokens": tokens, "hkv": hkv, "d": d, "page": page, "skip": skip,
            "decode": decode}


def _attend4(name, batch, lo, hi, drafts=1, hq=48, hkv=8, d=128, page=64, cap=0.0, lse=False):
    return {"name": name, "op": "attend4", "batch": batch, "lo": lo, "hi": hi, "drafts": drafts, "hq": hq, "hkv": hkv,
            "d": d, "page": page, "cap": cap, "lse": lse}


def listed():
    return [
        # One decode step of 32 far sequences, half of each head rotated by neighbours: latency.
        _rope("rope_decode32_part", 32, hq=48, rot=64, inter=True, norm=False, scaling="yarn", far=1 << 20, decode=True),
        # Prompts of a prefill step whose attention computes in bf16: Mixtral's heads, with norms.
        _rope("rope_prefill8192", 8192),
        # One decode step into the FP8 cache, static scales: Grok-1's heads, latency.
        _write("ropewrite_decode32", 32, norm=False, scales="head", decode=True),
        # A padded chunk of a prompt: one shared key/value head, small heads and pages, a part of each head rotated.
        _write("ropewrite_chunk1999_d64", 1999, hq=16, hkv=1, d=64, rot=32, page=16, scaling="linear", far=30000, skip=77),
        # The prompts of the prefill benchmark: 32 sequences of 1024 tokens, scales found as they are written.
        _write("ropewrite_prefill32768", 32768, scaling="wave"),
        # Pages and slots of one decode step of 256 sequences.
        _pages("pages_decode256", 256, 4096, 1, 1, pad=0),
        # A step that mixes decoding with prompts, padded, whose pool runs out on the last sequences.
        _pages("pages_mixed1024", 1024, 2000, 1, 200, page=16, pad=999, short=True),
        # One decode step's keys and values into 4 bits and back: latency.
        _rows4("rows4_decode32", 32, decode=True),
        # The prefill benchmark's prompts into 4 bits, and read back for a layer that computes in bf16.
        _rows4("rows4_prefill32768", 32768),
        # One user with a conversation behind them: the smallest step, latency.
        _attend4("attend4_b1_4000", 1, 4000, 4000),
        # Drafted tokens on trial: 24 sequences of 4 tokens each, one shared key/value head, small heads and pages, capped.
        _attend4("attend4_b24_drafts4_mqa_d64", 24, 0, 5001, drafts=4, hq=16, hkv=1, d=64, page=16, cap=30.0, lse=True),
        # Mixtral's heads, 64 long contexts: the largest.
        _attend4("attend4_b64_16384", 64, 8192, 16384, hq=32, lse=True),
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
    op = rng.choice(["rope", "rope_write", "pages", "rows4", "attend4", "attend4"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    hq, hkv = rng.choice([(48, 8), (32, 8), (40, 8), (8, 8), (16, 1), (28, 4)])
    if op == "pages":
        batch = _spread(rng, 1, 4096)
        new_hi = rng.choice([1, 5, _spread(rng, 1, max(1, min(8192, 65536 // batch)))])
        return {"op": op, "batch": batch, "ctx": _spread(rng, 1, max(16, min(32768, 4000000 // batch))),
                "new_lo": rng.choice([0, 1, new_hi]), "new_hi": new_hi, "page": page, "pad": rng.choice([0, 13, 1000]),
                "short": rng.random() < 0.25}
    if op == "rows4":
        tokens = _spread(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "hkv": hkv, "d": d, "page": page, "skip": rng.choice([0, tokens // 7]),
                "decode": tokens <= 512 and rng.random() < 0.5}
    if op == "attend4":
        batch, drafts = _spread(rng, 1, 256), rng.choice([1, 1, 2, 5])
        hi = _spread(rng, drafts, min(16384, max(64, 16384 * 64 // (batch * drafts))))
        return {"op": op, "batch": batch, "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "drafts": drafts, "hq": hq,
                "hkv": hkv, "d": d, "page": page, "cap": rng.choice([0.0, 0.0, 30.0]), "lse": rng.random() < 0.5}
    tokens = _spread(rng, 1, 32768)
    case = {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4, d - 16]),
            "inter": rng.random() < 0.4, "norm": rng.random() < 0.5,
            "scaling": rng.choice(["none", "linear", "base", "yarn", "wave"]), "far": rng.choice([4096, 131072, 1 << 20]),
            "decode": tokens <= 512 and rng.random() < 0.5}
    if op == "rope_write":
        case.update(page=page, scales=rng.choice(["head", "token"]), skip=rng.choice([0, tokens // 7]))
    return case


def _even(n, lo, hi):
    """n whole numbers evenly spread over lo..hi (a seed only changes their order)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _ceil(a, b):
    return -(-a // b)


def _requests(case):
    """(tokens in the cache, new tokens) of each sequence; a seed only changes their order."""
    b = case["batch"]
    new = _even(b, case["new_lo"], case["new_hi"])
    return list(zip(_even(b, case["ctx"] // 2, case["ctx"]), new[b // 2:] + new[:b // 2]))


def _taken(case):
    """Pages that the new tokens need."""
    return sum(_ceil(n + m, case["page"]) - _ceil(n, case["page"]) for n, m in _requests(case))


def work(case):
    op = case["op"]
    if op == "pages":
        t, b = sum(n for _, n in _requests(case)) + case["pad"], case["batch"]
        # lengths in and out twice, five numbers a token, an old page of each sequence, new pages to and fro
        n = 4 * (5 * b + 5 * t) + 4 * b + 16 * _taken(case)
        return {"bytes": n, "flops": 4 * t}
    if op == "rows4":
        t, hkv, d = case["tokens"], case["hkv"], case["d"]
        live = t - case["skip"]
        # write: bf16 in, codes and scales out; read: the same the other way round
        return {"bytes": live * hkv * 4 * d + 2 * live * hkv * (d + 8) + t * hkv * 4 * d + 8 * t,
                "flops": 12 * live * hkv * d}
    if op == "attend4":
        b, m, hq, hkv, d, page = (case[n] for n in ("batch", "drafts", "hq", "hkv", "d", "page"))
        lens = [max(n, m) for n in _even(b, case["lo"], case["hi"])] if m > 1 else _even(b, case["lo"], case["hi"])
        rows = [n - j for n in lens for j in range(m)]
        n = sum(lens) * hkv * (d + 8) + 4 * b * m * hq * d + (4 * b * m * hq if case["lse"] else 0)
        return {"bytes": n + 4 * sum(_ceil(x, page) for x in lens) + 8 * b * m, "flops": 4 * hq * d * sum(rows)}
    t, hq, hkv, d = (case[n] for n in ("tokens", "hq", "hkv", "d"))
    flops = t * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))
    weights = 4 * d if case["norm"] else 0
    if op == "rope":
        return {"bytes": 4 * t * (hq + hkv) * d + 4 * t + 4 * case["rot"] + weights, "flops": flops}
    live = t - case["skip"]
    scale = 8 if case["scales"] == "token" else 0
    n = 4 * t * hq * d + live * hkv * (4 * d + 2 * d + scale) + 8 * t + 4 * case["rot"] + weights
    return {"bytes": n + (0 if scale else 8 * hkv), "flops": flops + 4 * live * hkv * d}


# ---------------------------------------------------------------- inputs
# What a model's configuration says of its rotation: the base, and how it is stretched for long contexts.
BASE = {"none": 10000.0, "linear": 10000.0, "base": 10000.0, "yarn": 150000.0, "wave": 500000.0}
STRETCH = {"linear": dict(factor=4.0), "base": dict(factor=8.0), "yarn": dict(factor=32.0, original_len=4096),
           "wave": dict(factor=8.0, original_len=8192)}


def _positions(case, gen):
    """Decoding: anywhere up to `far`. Else prompts of 1024 tokens (the last one shorter), each from a start of its own."""
    t, far = case["tokens"], case["far"]
    if case["decode"]:
        return torch.randint(0, far, (t,), generator=gen, device="cuda", dtype=torch.int32)
    i = torch.arange(t, device="cuda")
    start = torch.randint(0, max(1, far - 1024), (t // 1024 + 1,), generator=gen, device="cuda")
    return (start[i // 1024] + i % 1024).to(torch.int32)


def _slots(t, page, skip, decode, gen):
    """-> (slots, pages of the cache)"""
    pages = t + 3 if decode else _ceil(t, page) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    if decode:  # every sequence writes into a page of its own
        slots = order[:t] * page + torch.randint(0, page, (t,), generator=gen, device="cuda")
    else:
        i = torch.arange(t, device="cuda")
        slots = order[i // page] * page + i % page
    if skip:
        slots[torch.randperm(t, generator=gen, device="cuda")[:skip]] = -1
    return slots.to(torch.int32), pages


def _activations(t, width, d, gen):
    """A fused projection's output: normal, a few channels of each head stronger than the others."""
    x = torch.randn(t, width // d, d, generator=gen, device="cuda")
    x *= 1.0 + 3.0 * (torch.rand(1, width // d, d, generator=gen, device="cuda") > 0.95)
    return x.to(torch.bfloat16).view(t, width)


def _prepare_rope(case, gen):
    t, hq, hkv, d = (case[n] for n in ("tokens", "hq", "hkv", "d"))
    qkv = _activations(t, (hq + 2 * hkv) * d, d, gen)
    s = SimpleNamespace(case=case, positions=_positions(case, gen), q=qkv[:, :hq * d].unflatten(1, (hq, d)),
                        k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                        v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), q_weight=None, k_weight=None,
                        q_out=torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"),
                        k_out=torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda"))
    if case["norm"]:
        s.q_weight, s.k_weight = (
            (1.0 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))
    if case["op"] == "rope_write":
        s.slots, s.pages = _slots(t, case["page"], case["skip"], case["decode"], gen)
        # one page more than the cache has: where the plain form puts the tokens that are skipped
        shape = (s.pages + 1, hkv, case["page"])
        s.k_all, s.v_all = (torch.randn(*shape, d, generator=gen, device="cuda").mul_(100.0).to(torch.float8_e4m3fn)
                            for _ in range(2))
        token = case["scales"] == "token"
        s.k_scale_all, s.v_scale_all = (
            0.02 + 0.02 * torch.rand(shape if token else (hkv,), generator=gen, device="cuda") for _ in range(2))
        s.k_cache, s.v_cache = s.k_all[:s.pages], s.v_all[:s.pages]
        s.k_scale, s.v_scale = (x[:s.pages] if token else x for x in (s.k_scale_all, s.v_scale_all))
    if own:  # the frequencies are laid out once, when the model is loaded
        import w4a8_moe_gb300 as lib

        scaling = case["scaling"]
        s.rope = lib.rope_table(case["rot"], base=BASE[scaling], scaling=None if scaling == "none" else scaling,
                                **STRETCH.get(scaling, {}))
    else:
        s.freqs, s.magnitude = _frequencies(case["rot"], case["scaling"])
        s.freqs = torch.tensor(s.freqs, dtype=torch.float64, device="cuda")
    return s


def _prepare_pages(case, gen):
    b, page = case["batch"], case["page"]
    requests = torch.tensor(_requests(case), dtype=torch.int32, device="cuda")
    lens, new = requests[torch.randperm(b, generator=gen, device="cuda")].t().contiguous()
    most = _ceil(case["ctx"] + case["new_hi"], page) + 1
    used = (lens.long() + page - 1) // page
    first = torch.cumsum(used, 0) - used
    need = _taken(case)
    free = need - need // 8 if case["short"] else need + need // 4 + 1
    held = int(used.sum())
    perm = torch.randperm(held + free, generator=gen, device="cuda").to(torch.int32)
    rank = torch.arange(most, device="cuda")[None]
    table = torch.where(rank < used[:, None], perm[(first[:, None] + rank).clamp(max=held + free - 1)], -1)
    stack = torch.full((held + free,), -1, dtype=torch.int32, device="cuda")
    stack[:free] = perm[held:]
    return SimpleNamespace(case=case, lens=lens, new=new, table=table.to(torch.int32), stack=stack,
                           count=torch.tensor([free], dtype=torch.int32, device="cuda"),
                           capacity=sum(n for _, n in _requests(case)) + case["pad"],
                           ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))


def _prepare_rows4(case, gen):
    t, hkv, d, page = (case[n] for n in ("tokens", "hkv", "d", "page"))
    kv = _activations(t, 2 * hkv * d, d, gen)
    slots, pages = _slots(t, page, case["skip"], case["decode"], gen)
    shape = (pages + 1, hkv, page)
    k_all, v_all = (torch.randint(0, 256, (*shape, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
                    for _ in range(2))
    k_s, v_s = (torch.rand(*shape, 2, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    return SimpleNamespace(case=case, pages=pages, slots=slots, k=kv[:, :hkv * d].unflatten(1, (hkv, d)),
                           v=kv[:, hkv * d:].unflatten(1, (hkv, d)), k_all=k_all, v_all=v_all, k_scale_all=k_s,
                           v_scale_all=v_s, k_cache=k_all[:pages], v_cache=v_all[:pages], k_scale=k_s[:pages],
                           v_scale=v_s[:pages], k_out=torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda"),
                           v_out=torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda"))


def _codes4(gen, pages, hkv, page, d):
    """A filled cache: 4-bit codes, two to a byte, with each row's step and least value. Normal values, a few channels of
    each head stronger than the others and off centre, tokens of differing strength."""
    x = torch.randn(pages, hkv, page, d, generator=gen, device="cuda")
    x *= 1.0 + 3.0 * (torch.rand(1, hkv, 1, d, generator=gen, device="cuda") > 0.95)
    x += 0.5 * torch.randn(1, hkv, 1, d, generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn(pages, hkv, page, 1, generator=gen, device="cuda"))
    least = x.amin(-1).to(torch.bfloat16)
    step = ((x.amax(-1) - least.float()) / 15.0).to(torch.bfloat16)
    x -= least.float()[..., None]
    x /= step.float()[..., None]
    c = x.round_().clamp_(0, 15).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([step, least], -1)


def _prepare_attend4(case, gen):
    b, m, hq, hkv, d, page = (case[n] for n in ("batch", "drafts", "hq", "hkv", "d", "page"))
    lens = torch.tensor(_even(b, case["lo"], case["hi"]), device="cuda")
    if m > 1:
        lens = lens.clamp(min=m)
    lens = lens[torch.randperm(b, generator=gen, device="cuda")]
    most = max(1, _ceil(case["hi"], page))
    used = (lens + page - 1) // page
    pages = int(used.sum()) + 2
    order = torch.randperm(pages, generator=gen, device="cuda")
    rank = torch.arange(most, device="cuda")[None]
    first = torch.cumsum(used, 0) - used
    table = torch.where(rank < used[:, None], order[(first[:, None] + rank).clamp(max=pages - 1)], -1)
    k_cache, k_scale = _codes4(gen, pages, hkv, page, d)
    v_cache, v_scale = _codes4(gen, pages, hkv, page, d)
    # what lies behind a sequence's last token in its last page is whatever was there: here rows that are no numbers
    last = table.gather(1, (used[:, None] - 1).clamp(min=0))[:, 0]
    last = torch.where(used > 0, last, order[-1])  # the last of the order belongs to nobody
    dead = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    dead[last] = (used > 0)[:, None] & (torch.arange(page, device="cuda")[None] >= (lens - (used - 1) * page)[:, None])
    for x in (k_scale, v_scale):
        x.masked_fill_(dead[:, None, :, None], float("nan"))
    t = b * m
    qkv = (torch.randn(t, (hq + 2 * hkv) * d, generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    seqs = torch.arange(b, device="cuda").repeat_interleave(m)
    seen = lens[seqs] - (m - 1) + torch.arange(m, device="cuda").repeat(b)  # each draft sees those before it
    s = SimpleNamespace(case=case, q=qkv[:, :hq * d].unflatten(1, (hq, d)), k_cache=k_cache, v_cache=v_cache,
                        k_scale=k_scale, v_scale=v_scale, table=table.to(torch.int32), seen=seen.to(torch.int32),
                        seqs=seqs.to(torch.int32), scale=d ** -0.5,
                        out=torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"),
                        lse=torch.empty(t, hq, device="cuda") if case["lse"] else None, ws=None)
    if own:  # a decoding program keeps one workspace
        import w4a8_moe_gb300 as lib

        s.ws = torch.zeros(lib.kv4_attention_workspace_size(t, hq, hkv, d, most, page), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "rope_write": _prepare_rope, "pages": _prepare_pages, "rows4": _prepare_rows4,
            "attend4": _prepare_attend4}[case["op"]](case, gen)


# ---------------------------------------------------------------- the framework's calls
def _written(s):
    out = [s.q_out, s.k_cache, s.v_cache]
    return out + [s.k_scale, s.v_scale] if s.case["scales"] == "token" else out


def _run_own(s):
    import w4a8_moe_gb300 as lib

    c = s.case
    if c["op"] == "rope":
        return list(lib.qk_norm_rope(s.q, s.k, s.positions, s.rope, s.q_weight, s.k_weight, eps=1e-6,
                                     interleaved=c["inter"], q_out=s.q_out, k_out=s.k_out))
    if c["op"] == "rope_write":
        lib.kv8_norm_rope_write(s.q, s.k, s.v, s.positions, s.slots, s.rope, s.k_cache, s.v_cache, s.k_scale, s.v_scale,
                                s.q_weight, s.k_weight, eps=1e-6, interleaved=c["inter"], q_out=s.q_out)
        return _written(s)
    if c["op"] == "pages":  # a step's pages are taken and given back, so that a pass leaves the pool as it found it
        step = lib.kv_pages_extend(s.lens, s.new, s.table, s.stack, s.count, c["page"], s.capacity, ws=s.ws)
        after = lib.kv_pages_truncate(step.lens, s.lens, s.table, s.stack, s.count, c["page"], ws=s.ws)
        return [step.starts, step.seqs, step.positions, step.seen, step.slots, step.lens, after, s.table, s.stack, s.count]
    if c["op"] == "rows4":
        lib.kv4_write(s.k, s.v, s.slots, s.k_cache, s.v_cache, s.k_scale, s.v_scale)
        k, v = lib.kv4_read(s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.slots, k_out=s.k_out, v_out=s.v_out)
        return [k, v, s.k_scale, s.v_scale]
    out, lse = lib.kv4_attention(s.q, s.k_cache, s.v_cache, s.k_scale, s.v_scale, s.table, s.seen,
                                 seqs=s.seqs if c["drafts"] > 1 else None, sm_scale=s.scale, logit_cap=c["cap"], out=s.out,
                                 lse=s.lse, ws=s.ws)
    return [out] if lse is None else [out, lse]


# ---------------------------------------------------------------- plain forms
def _frequencies(rot, scaling):
    """Radians per position of each pair, and what the rotated values are multiplied by."""
    base, p = BASE[scaling], STRETCH.get(scaling, {})
    f, n = p.get("factor", 1.0), rot // 2
    if scaling == "base":
        base = base * f ** (rot / max(1, rot - 2))
    freqs = [base ** (-2.0 * i / rot) for i in range(n)]
    if scaling == "linear":
        return [x / f for x in freqs], 1.0
    if scaling == "yarn":  # pairs that turn often over the original length stay, those that turn less than once stretch
        def pair_of(turns):
            return rot * math.log(p["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
        hi = hi + 0.001 if lo == hi else hi
        ramp = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(n)]
        return [x * (1 - r) + x / f * r for x, r in zip(freqs, ramp)], 0.1 * math.log(f) + 1.0
    if scaling == "wave":  # the same by wavelength: a quarter of the original length and less stays, all of it stretches
        out = []
        for x in freqs:
            r = min(1.0, max(0.0, (p["original_len"] * x / (2 * math.pi) - 1.0) / (4.0 - 1.0)))
            out.append(x * r + x / f * (1 - r))
        return out, 1.0
    return freqs, 1.0


def _plain_rotate(s, x, weight):
    c = s.case
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = s.positions.double()[:, None] * s.freqs
    cos, sin = (f(angle).float()[:, None] * s.magnitude for f in (torch.cos, torch.sin))
    rot = c["rot"]
    if c["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    return [_plain_rotate(s, x, w).to(torch.bfloat16) for x, w in ((s.q, s.q_weight), (s.k, s.k_weight))]


def _plain_rope_write(s):
    page = s.case["page"]
    slots = torch.where(s.slots >= 0, s.slots, s.pages * page).long()
    at, off = slots // page, slots % page
    s.q_out.copy_(_plain_rotate(s, s.q, s.q_weight))
    k = _plain_rotate(s, s.k, s.k_weight)
    for x, cache, scale in ((k, s.k_all, s.k_scale_all), (s.v.float(), s.v_all, s.v_scale_all)):
        if s.case["scales"] == "token":
            f = x.abs().amax(-1)
            f = f / torch.full_like(f, E4M3_MAX)
            f = torch.where(f == 0, 1.0, f)
            scale[at, :, off] = f
        else:
            f = scale[None]
        codes = (x / f[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache.view(torch.uint8)[at, :, off] = codes.view(torch.uint8)
    return _written(s)


def _plain_pages(s):
    page, cap = s.case["page"], s.capacity
    lens, new = s.lens.long(), s.new.long()
    used = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - used
    before = torch.cumsum(need, 0) - need
    count = s.count.long()
    fits = (need == 0) | (before + need <= count)
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(new, 0)])
    t = torch.arange(cap, device="cuda")
    there = t < starts[-1]
    seq = torch.searchsorted(starts, t, right=True).sub(1).clamp(max=lens.numel() - 1)
    pos = lens[seq] + t - starts[seq]
    rank = torch.arange(s.table.shape[1], device="cuda")[None]
    fresh = (rank >= used[:, None]) & (rank < (used + need)[:, None]) & fits[:, None]
    at = (count - 1 - before[:, None] - (rank - used[:, None])).clamp(0, s.stack.numel() - 1)
    s.table.copy_(torch.where(fresh, s.stack[at], s.table))
    slot = s.table[seq, (pos // page).clamp(max=s.table.shape[1] - 1)].long() * page + pos % page
    i32 = torch.int32
    grown = torch.where(fits, lens + new, lens).to(i32)
    taken = torch.where(fits, need, 0).sum()
    s.count.sub_(taken)
    step = [starts.to(i32), torch.where(there, seq, -1).to(i32), torch.where(there, pos, 0).to(i32),
            torch.where(there & fits[seq], pos + 1, 0).to(i32), torch.where(there & fits[seq], slot, -1).to(i32), grown]
    # and back: the pages behind the kept tokens, the first sequence's first page on top of the stack
    give = torch.where(fits, need, 0)
    ahead = torch.cumsum(give, 0) - give
    back = (rank >= used[:, None]) & (rank < (used + give)[:, None])
    to = s.count.long() + taken - 1 - ahead[:, None] - (rank - used[:, None])
    to = torch.where(back, to, s.stack.numel())
    s.stack.copy_(torch.cat([s.stack, s.stack[:1]]).scatter(0, to.flatten(), s.table.flatten())[:-1])
    s.count.add_(taken)
    return step + [s.lens.clone(), s.table, s.stack, s.count]


def _plain_rows4(s):
    page = s.case["page"]
    slots = torch.where(s.slots >= 0, s.slots, s.pages * page).long()
    at, off = slots // page, slots % page
    outs = []
    for x, cache, scale in ((s.k, s.k_all, s.k_scale_all), (s.v, s.v_all, s.v_scale_all)):
        x = x.float()
        least = x.amin(-1)
        step = (x.amax(-1) * 0.5 - least * 0.5) / torch.full_like(least, 7.5)
        pair = torch.stack([step, least], -1).to(torch.bfloat16)
        step = pair[..., 0].float()
        c = torch.where(step[..., None] > 0, (x - least[..., None]) / step[..., None], 0.0)
        c = c.round().clamp(0, 15).to(torch.uint8)
        cache[at, :, off] = c[..., 0::2] | (c[..., 1::2] << 4)
        scale[at, :, off] = pair
        c, pair = cache[at, :, off], scale[at, :, off].float()
        y = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() * pair[..., :1] + pair[..., 1:]
        outs.append(torch.where((s.slots >= 0)[:, None, None], y, 0.0).to(torch.bfloat16))
    return outs + [s.k_scale, s.v_scale]


def _plain_keys4(cache, scale, pages):
    """[..., pages] of a table -> fp32 [kv heads, ..., keys, head dim]."""
    c, f = cache[pages], scale[pages].float()
    x = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() * f[..., :1] + f[..., 1:]
    return x.movedim(-3, 0).flatten(-3, -2)


def _plain_attend4(s):
    c = s.case
    m, hq, hkv, d, cap = (c[n] for n in ("drafts", "hq", "hkv", "d", "cap"))
    b, group = c["batch"], hq // hkv
    # [kv heads, batch, drafts * group, d]
    q = s.q.float().reshape(b, m, hkv, group, d).permute(2, 0, 1, 3, 4).reshape(hkv, b, m * group, d)
    table = s.table.clamp(min=0).long()
    k = _plain_keys4(s.k_cache, s.k_scale, table)
    i = torch.arange(k.shape[2], device="cuda")
    live = i < s.seen.view(b, m)[:, -1:]  # [batch, keys]: of the last draft, which sees all that exist
    sees = (i < s.seen[:, None]).view(b, m, 1, -1).expand(b, m, group, i.numel()).reshape(b, m * group, -1)
    x = torch.matmul(q, torch.where(live[None, ..., None], k, 0.0).transpose(-1, -2)) * s.scale
    del k
    if cap:
        x = cap * torch.tanh(x / cap)
    x = torch.where(sees, x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    w = torch.exp(x - top)
    del x
    total = w.sum(-1, keepdim=True)
    v = torch.where(live[None, ..., None], _plain_keys4(s.v_cache, s.v_scale, table), 0.0)
    out = torch.matmul(w, v)
    out = torch.where(total > 0, out / torch.where(total > 0, total, 1.0), 0.0)

    def order(y):
        return y.reshape(hkv, b, m, group, -1).permute(1, 2, 0, 3, 4).reshape(b * m, hq, -1)

    out = order(out).to(torch.bfloat16)
    return [out, order(top + torch.log(total))[..., 0]] if c["lse"] else [out]


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "rope_write": _plain_rope_write, "pages": _plain_pages, "rows4": _plain_rows4,
            "attend4": _plain_attend4}[state.case["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _exact_rotate(s, x, weight, freqs, magnitude):
    """As a product of complex numbers, token by token's own angle."""
    c = s.case
    rot, x = c["rot"], x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * weight.double()
    angle = s.positions.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
    head = x[..., :rot].contiguous()
    if c["inter"]:
        y = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2))) * turn).flatten(-2)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _round64(x):
    """x to the nearest E4M3 value, ties to even, saturating."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rope(s):
    c = s.case
    freqs, magnitude = _frequencies(c["rot"], c["scaling"])
    q, k = (_exact_rotate(s, x, w, freqs, magnitude) for x, w in ((s.q, s.q_weight), (s.k, s.k_weight)))
    if c["op"] == "rope":
        return [q, k]
    page, token = c["page"], c["scales"] == "token"
    keep = torch.nonzero(s.slots >= 0)[:, 0]
    slots = s.slots[keep].long()
    caches, scales = [], []
    for x, cache, scale in ((k, s.k_cache, s.k_scale), (s.v, s.v_cache, s.v_scale)):
        vals = cache.double().permute(0, 2, 1, 3).reshape(s.pages * page, c["hkv"], c["d"])
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
        caches.append(vals.reshape(s.pages, page, c["hkv"], -1).permute(0, 2, 1, 3))
    return [q] + caches + scales


def _exact_rows4(s):
    page, hkv = s.case["page"], s.case["hkv"]
    keep = torch.nonzero(s.slots >= 0)[:, 0]
    slots = s.slots[keep].long()
    outs, scales = [], []
    for x, scale in ((s.k, s.k_scale), (s.v, s.v_scale)):
        x = x.double()[keep]
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        step = (hi - lo) / 15
        rows = scale.double().transpose(1, 2).reshape(s.pages * page, hkv, 2)
        rows[slots] = torch.cat([step, lo], -1)
        scales.append(rows.reshape(s.pages, page, hkv, 2).transpose(1, 2))
        step = step.to(torch.bfloat16).double()  # codes stand for multiples of the step as it is kept
        n = torch.where(step > 0, (x - lo) / torch.where(step > 0, step, 1.0), 0.0)
        y = torch.zeros(s.case["tokens"], hkv, s.case["d"], dtype=torch.float64, device="cuda")
        y[keep] = lo + step * torch.round(n).clamp(0, 15)
        outs.append(y)
    return outs + scales


def _exact_attend4(s):
    c = s.case
    hq, hkv, d, page = (c[n] for n in ("hq", "hkv", "d", "page"))
    t = c["batch"] * c["drafts"]
    outs = torch.zeros(t, hq, d, dtype=torch.float64, device="cuda")
    lses = torch.full((t, hq), -torch.inf, dtype=torch.float64, device="cuda")
    seen, seqs = s.seen.tolist(), s.seqs.tolist()
    for i in range(t):
        n = seen[i]
        if n == 0:
            continue
        pages = s.table[seqs[i], :_ceil(n, page)].long()
        k, v = (((((x[pages][..., None] >> torch.tensor([0, 4], device="cuda", dtype=torch.uint8)) & 15).flatten(-2).double()
                  * f[pages][..., :1].double() + f[pages][..., 1:].double()).transpose(0, 1).reshape(hkv, -1, d))[:, :n]
                for x, f in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale)))
        x = s.q[i].double().reshape(hkv, hq // hkv, d) @ k.transpose(1, 2) * s.scale
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        z = torch.logsumexp(x, -1)
        lses[i] = z.reshape(hq)
        outs[i] = (torch.exp(x - z[..., None]) @ v).reshape(hq, d)
    return [outs, lses] if c["lse"] else [outs]


def exact(case, seed):
    if case["op"] == "pages":  # whole numbers, which are compared as they are
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "rope_write": _exact_rope, "rows4": _exact_rows4, "attend4": _exact_attend4}[case["op"]](s)
