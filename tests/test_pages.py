"""Page tables and slots built on the GPU against a plain list of pages, and a serving step that uses them."""
import numpy as np
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu

W4A8_ERR_INDEX, W4A8_ERR_PAGES = 8, 9
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


def ceil(a, b):
    return -(-a // b)


class Pool:
    """Tables and the stack of free pages as plain lists."""

    def __init__(self, lens, page, most, spare, seed=0):
        rng = np.random.default_rng(seed)
        need = [ceil(n, page) for n in lens]
        self.page, self.most, self.num = page, most, sum(need) + spare
        order = rng.permutation(self.num).tolist()
        self.lens = list(lens)
        self.rows = []
        for n in need:
            self.rows.append([order.pop() for _ in range(n)])
        self.stack = order
        self.stale = np.full((len(lens), most), -7)
        for b, r in enumerate(self.rows):
            self.stale[b, :len(r)] = r
        assert len(order) == spare

    def gpu(self):
        stack = np.full(self.num, -9)
        stack[:len(self.stack)] = self.stack
        make = lambda x: torch.tensor(np.asarray(x), dtype=I32, device="cuda")  # noqa: E731
        return make(self.lens), make(self.stale), make(stack), make([len(self.stack)])

    def extend(self, new, capacity):
        """-> (starts, tokens [(seq, position, seen, slot)], error)"""
        starts, tokens, err, need_so_far = [0], [], 0, 0
        have = len(self.stack)
        for b, n in enumerate(new):
            n = max(n, 0)
            total = starts[-1] + n
            ok = new[b] >= 0 and self.lens[b] + n <= self.most * self.page
            need = ceil(self.lens[b] + n, self.page) - len(self.rows[b]) if ok else 0
            need_so_far += need
            if not ok or total > capacity:
                err, fits = W4A8_ERR_INDEX, False
            else:
                fits = need == 0 or need_so_far <= have
            if need and need_so_far > have:
                err = err or W4A8_ERR_PAGES
            if fits:
                for _ in range(need):
                    self.rows[b].append(self.stack.pop())
                    self.stale[b, len(self.rows[b]) - 1] = self.rows[b][-1]
            for i in range(min(n, capacity)):
                p = self.lens[b] + i
                tokens.append((b, p, p + 1, self.rows[b][p // self.page] * self.page + p % self.page) if fits
                              else (b, p, 0, -1))
            if fits:
                self.lens[b] += n
            starts.append(total)
        return [min(s, capacity) for s in starts], tokens[:capacity], err

    def truncate(self, keep):
        gone = []
        for b, n in enumerate(keep):
            k = ceil(n, self.page)
            gone += self.rows[b][k:]
            del self.rows[b][k:]
            self.lens[b] = n
        self.stack += gone[::-1]


def same_pool(p, table, stack, count, lens):
    assert int(count) == len(p.stack)
    assert stack.tolist()[:len(p.stack)] == p.stack
    assert np.array_equal(table.cpu().numpy(), p.stale)
    assert lens.tolist() == p.lens


def extend_and_compare(lib, p, state, new, capacity, ws, in_place=True):
    lens, table, stack, count = state
    out = None
    if in_place:
        b = len(new)
        out = lib.PageStep(*[torch.full((n,), -77, dtype=I32, device="cuda") for n in [b + 1] + [capacity] * 4], lens)
    step = lib.kv_pages_extend(lens, torch.tensor(new, dtype=I32, device="cuda"), table, stack, count, p.page, capacity,
                               out=out, ws=ws)
    starts, tokens, err = p.extend(new, capacity)
    assert step.starts.tolist() == starts
    tokens += [(-1, 0, 0, -1)] * (capacity - len(tokens))
    for got, want in zip((step.seqs, step.positions, step.seen, step.slots), zip(*tokens)):
        assert got.tolist() == list(want)
    same_pool(p, table, stack, count, step.lens)
    assert lib.w4a8_device_error(ws) == err
    return step


def workspace(lib):
    return torch.zeros(lib.kv_pages_workspace_size(), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("batch,page,longest,new,pad", [
    (1, 16, 1, 1, 0), (1, 64, 5000, 4000, 3), (5, 16, 70, 40, 1), (32, 64, 500, 1, 0), (256, 32, 300, 1, 44),
    (257, 16, 40, 9, 0), (300, 256, 2000, 300, 1000), (1000, 16, 10, 2, 7), (4096, 16, 33, 20, 5), (4096, 128, 200, 1, 0),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_and_truncate(lib, batch, page, longest, new, pad, in_place):
    """A few steps of growing and shrinking, some sequences idle, some starting from nothing, some finished."""
    rng = np.random.default_rng(batch + page)
    lens = rng.integers(0, longest + 1, batch).tolist()
    most = ceil(longest + 4 * new, page) + 1
    p = Pool(lens, page, most, spare=batch * ceil(4 * new, page) + batch, seed=batch)
    state = p.gpu()
    ws = workspace(lib)
    for _ in range(3):
        add = rng.integers(0, new + 1, batch)
        add[rng.random(batch) < 0.2] = 0
        add = add.tolist()
        step = extend_and_compare(lib, p, state, add, max(sum(add) + pad, 1), ws, in_place)
        state = (step.lens, *state[1:])
        keep = [0 if rng.random() < 0.1 else int(rng.integers(max(0, n - new - page), n + 1)) for n in p.lens]
        after = lib.kv_pages_truncate(state[0], torch.tensor(keep, dtype=I32, device="cuda"), *state[1:], page,
                                      out=state[0] if in_place else None, ws=ws)
        p.truncate(keep)
        same_pool(p, *state[1:], after)
        assert lib.w4a8_device_error(ws) == 0
        state = (after, *state[1:])


@pytest.mark.parametrize("batch", range(4084, 4097))
def test_largest_batches(lib, batch):
    """Their sums take a block's shared memory past the 48 KB that need no asking for."""
    p = Pool([b % 17 for b in range(batch)], 16, 3, spare=batch, seed=batch)
    state = p.gpu()
    ws = workspace(lib)
    new = [b % 3 for b in range(batch)]
    step = extend_and_compare(lib, p, state, new, sum(new) + 1, ws)
    keep = [n // 2 for n in p.lens]
    after = lib.kv_pages_truncate(step.lens, torch.tensor(keep, dtype=I32, device="cuda"), *state[1:], 16, ws=ws)
    p.truncate(keep)
    same_pool(p, *state[1:], after)
    assert lib.w4a8_device_error(ws) == 0


def test_truncating_what_was_extended_restores_the_stack(lib):
    p = Pool([3, 0, 64, 65, 200], 16, 40, spare=30)
    lens, table, stack, count = p.gpu()
    before = stack.clone(), count.clone()
    step = lib.kv_pages_extend(lens, torch.tensor([40, 1, 0, 100, 7], dtype=I32, device="cuda"), table, stack, count, 16, 200)
    assert int(count) < int(before[1])
    back = lib.kv_pages_truncate(step.lens, lens, table, stack, count, 16)
    assert torch.equal(stack, before[0]) and torch.equal(count, before[1]) and torch.equal(back, lens)


@pytest.mark.parametrize("batch", [3, 40, 700])
def test_pool_runs_out(lib, batch):
    """Sequences past the end of the pool get nothing and stay as they were; those that need no page go on."""
    p = Pool([15] * batch, 16, 8, spare=batch // 2)
    state = p.gpu()
    ws = workspace(lib)
    new = [2 if i % 3 else 1 for i in range(batch)]   # every third fits its last page
    step = extend_and_compare(lib, p, state, new, sum(new) + 5, ws)
    assert step.lens.tolist()[0] == 16
    new = [0] * batch
    new[-1] = 16 * 7
    extend_and_compare(lib, p, (step.lens, *state[1:]), new, 200, ws)


def test_too_long_too_many_and_negative(lib):
    """Each is refused alone, reported, and leaves the others right."""
    ws = workspace(lib)
    p = Pool([10, 100, 5, 33], 16, 8, spare=40)
    state = p.gpu()
    step = extend_and_compare(lib, p, state, [3, 29, 2, 2 ** 31 - 1], 60, ws)     # past the table, past everything
    step = extend_and_compare(lib, p, (step.lens, *state[1:]), [3, -4, 2, 1], 60, ws)
    step = extend_and_compare(lib, p, (step.lens, *state[1:]), [3, 4, 20, 1], 10, ws)   # the third does not fit, nor the last
    step = extend_and_compare(lib, p, (step.lens, *state[1:]), [1, 0, 0, 0], 1, ws)
    # a negative length: its tokens get nothing
    lens = step.lens.clone()
    lens[1] = -5
    table, stack, count = (x.clone() for x in state[1:])
    out = lib.kv_pages_extend(lens, torch.tensor([1, 2, 1, 1], dtype=I32, device="cuda"), table, stack, count, 16, 5, ws=ws)
    assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX
    assert out.lens.tolist()[1] == -5 and out.slots.tolist()[1:3] == [-1, -1] and out.seen.tolist()[1:3] == [0, 0]
    assert out.starts.tolist() == [0, 1, 3, 4, 5]


def test_broken_tables_and_stacks_are_reported(lib):
    ws = workspace(lib)
    for what in ("table", "stack", "many", "negative"):
        p = Pool([10, 20], 16, 8, spare=6)
        lens, table, stack, count = p.gpu()
        if what == "table":
            table[1, 1] = p.num
        elif what == "stack":
            stack[5] = -1
        else:
            count.fill_(p.num + 1 if what == "many" else -3)
        out = lib.kv_pages_extend(lens, torch.tensor([1, 20], dtype=I32, device="cuda"), table, stack, count, 16, 30, ws=ws)
        assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX, what
        slots = out.slots.tolist()
        assert all(-1 <= s < p.num * 16 for s in slots)
        if what == "table":
            assert slots[1:13] == [-1] * 12 and slots[13] >= 0
        lib.w4a8_device_error(ws)
    p = Pool([100, 20], 16, 8, spare=2)
    lens, table, stack, count = p.gpu()
    for keep in ([101, 5], [-1, 20]):   # only the second moves
        got = lib.kv_pages_truncate(lens, torch.tensor(keep, dtype=I32, device="cuda"), table, stack, count, 16, ws=ws)
        assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX
        assert got.tolist()[0] == 100
    assert int(count) == 3
    count.fill_(p.num - 1)   # a count that leaves no room
    before = stack.clone()
    got = lib.kv_pages_truncate(lens, torch.tensor([0, 0], dtype=I32, device="cuda"), table, stack, count, 16, ws=ws)
    assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX
    assert torch.equal(got, lens) and torch.equal(stack, before) and int(count) == p.num - 1


def test_strided_tables_and_guards(lib):
    """Rows of a larger table; nothing beside them or behind the outputs is touched."""
    p = Pool([10, 0, 47], 16, 6, spare=20)
    lens, table, stack, count = p.gpu()
    big = torch.full((3, 20), -5, dtype=I32, device="cuda")
    big[:, 7:13] = table
    ws = workspace(lib)
    extend_and_compare(lib, p, (lens, big[:, 7:13], stack, count), [30, 17, 1], 50, ws)
    assert bool((big[:, :7] == -5).all()) and bool((big[:, 13:] == -5).all())
    buf = torch.full((6, 300), -5, dtype=I32, device="cuda")
    out = lib.PageStep(buf[0, 100:104], *[buf[i, 100:117] for i in range(1, 5)], buf[5, 100:103])
    lib.kv_pages_extend(lens, torch.tensor([1, 2, 3], dtype=I32, device="cuda"), big[:, 7:13], stack, count, 16, 17, out=out, ws=ws)
    for row, n in zip(buf, (4, 17, 17, 17, 17, 3)):
        assert bool((row[:100] == -5).all()) and bool((row[100 + n:] == -5).all())


def test_captured_decoding_loop(lib):
    """One captured step, replayed: lengths, tables and the pool go on in device memory; another stream gives the same."""
    p = Pool([15, 0, 40, 31], 16, 12, spare=40)
    lens, table, stack, count = p.gpu()
    new = torch.ones(4, dtype=I32, device="cuda")
    ws = workspace(lib)
    out = lib.PageStep(*[torch.empty(n, dtype=I32, device="cuda") for n in (5, 6, 6, 6, 6)], lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.kv_pages_extend(lens, new, table, stack, count, 16, 6, out=out, ws=ws)
    for i in range(100):
        add = [1, 1, i % 2, 0 if i > 50 else 1]
        new.copy_(torch.tensor(add, dtype=I32))
        graph.replay()
        starts, tokens, err = p.extend(add, 6)
        assert err == 0 and out.starts.tolist() == starts
        assert out.slots.tolist() == [t[3] for t in tokens] + [-1] * (6 - len(tokens))
        same_pool(p, table, stack, count, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step = lib.kv_pages_extend(lens, new, table, stack, count, 16, 8, stream=side)
    back = lib.kv_pages_truncate(step.lens, torch.zeros_like(lens), table, stack, count, 16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    p.extend(add, 8)
    p.truncate([0] * 4)
    same_pool(p, table, stack, count, back)


def test_python_checks_raise_before_a_launch(lib):
    p = Pool([10, 0, 47], 16, 6, spare=20)
    lens, table, stack, count = p.gpu()
    new = torch.ones_like(lens)
    good = dict(lens=lens, new_lens=new, page_table=table, free_pages=stack, free_count=count, page_size=16, capacity=8)
    for change in (dict(lens=lens.long()), dict(new_lens=new[:2]), dict(page_table=table[:2]), dict(page_table=table.t()),
                   dict(free_pages=stack.long()), dict(free_count=count.expand(2)), dict(page_size=17), dict(capacity=0),
                   dict(new_lens=new.cpu()), dict(page_table=table[:, :0]), dict(ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, lib.W4A8Error)):
            lib.kv_pages_extend(**dict(good, **change))
    for args in ((lens, new[:2], table, stack, count, 16), (lens.float(), new, table, stack, count, 16),
                 (lens, new, table, stack, count, 8)):
        with pytest.raises((ValueError, lib.W4A8Error)):
            lib.kv_pages_truncate(*args)


# ---------------------------------------------------------------- a serving step of all of it
@pytest.mark.parametrize("bits,d,hq,hkv,page", [(8, 128, 12, 2, 16), (8, 64, 8, 8, 32), (4, 128, 12, 2, 16), (4, 64, 16, 1, 64)])
def test_serving_steps(lib, bits, d, hq, hkv, page):
    """Prompts, then decoding with drafted tokens of which some are rejected and sequences that end and begin: pages,
    rotation, cache and attention against the dense attention over what the caches hold, with exact rotations."""
    gen = torch.Generator(device="cuda").manual_seed(bits + d)
    rng = np.random.default_rng(bits + d)
    batch, most, pages = 4, 16, 60
    rope = lib.rope_table(d)
    kw = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
    if bits == 8:
        cache = ([torch.zeros(pages, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
                 + [torch.zeros(pages, hkv, page, device="cuda") for _ in range(2)])
    else:
        cache = ([torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
                 + [torch.zeros(pages, hkv, page, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    lens = torch.zeros(batch, dtype=I32, device="cuda")
    table = torch.full((batch, most), -1, dtype=I32, device="cuda")
    stack, count = torch.randperm(pages, generator=gen, device="cuda").to(I32), torch.tensor([pages], dtype=I32, device="cuda")
    ws = workspace(lib)
    history = [[] for _ in range(batch)]   # the rows (position, fp32 k, v) of each sequence as they went in
    for step_no in range(8):
        new = rng.integers(20, 60, batch) if step_no == 0 else rng.integers(0, 5, batch)
        cap = int(new.sum()) + 3
        step = lib.kv_pages_extend(lens, torch.tensor(new.tolist(), dtype=I32, device="cuda"), table, stack, count, page, cap, ws=ws)
        qkv = torch.randn(cap, hq + 2 * hkv, d, generator=gen, device="cuda").to(torch.bfloat16)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if bits == 8:
            q2 = lib.kv8_norm_rope_write(q, k, v, step.positions, step.slots, rope, *cache, kw, kw)
        else:
            q2, k2 = lib.qk_norm_rope(q, k, step.positions, rope, kw, kw)
            lib.kv4_write(k2, v, step.slots, *cache)
        seqs = step.seqs
        if bits == 8:
            rows = table[seqs.clamp(min=0).long()]
            out, _ = lib.kv8_prefix_attention(q2, *cache, None, 0, rows, step.seen)
        else:
            out, _ = lib.kv4_attention(q2, *cache, table, step.seen, seqs=seqs)
        read = lib.kv8_read if bits == 8 else lib.kv4_read
        kf, vf = (x.double() for x in lib.qk_norm_rope(k, v, step.positions, rope, kw)[:1] + (v,))
        for t, b in enumerate(seqs.tolist()):
            if b < 0:
                assert bool((out[t] == 0).all())
                continue
            pos = int(step.positions[t])
            assert pos == len(history[b])
            history[b].append((kf[t], vf[t]))
            # the sequence's keys as the cache gives them back, slot by slot of its table
            slots = (table[b, torch.arange(pos + 1, device="cuda") // page] * page
                     + torch.arange(pos + 1, device="cuda", dtype=I32) % page).to(I32)
            kc, vc = read(*cache, slots)
            for got, i in ((kc, 0), (vc, 1)):
                want = torch.stack([h[i] for h in history[b]])
                # within a step of the 8- or 4-bit format
                unit = want.abs().amax(-1, keepdim=True) if bits == 8 else want.amax(-1, keepdim=True) - want.amin(-1, keepdim=True)
                bound = want.abs() * 2.0 ** -4 + unit * 2.0 ** -8 if bits == 8 else unit / 15 * 0.6 + want.abs() * 2.0 ** -7
                assert bool(((got.double() - want).abs() <= bound + 1e-3 * unit).all())
            if t % 5:
                continue
            s = torch.einsum("hgd,nhd->hgn", q2[t].double().view(hkv, hq // hkv, d), kc.double()) * d ** -0.5
            ref = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vc.double()).reshape(hq, d)
            # kc and vc are rounded to bf16 (2^-8 of a value: scores of a few units move by a few times that, 2^-5 at most
            # here, and the weights with them), the output too
            mag = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vc.double().abs()).reshape(hq, d)
            ds = (torch.einsum("hgd,nhd->hgn", q2[t].double().abs().view(hkv, hq // hkv, d), kc.double().abs()) * d ** -0.5).amax(-1)
            tol = (2 * ds.reshape(hq, 1) * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10) * mag * 1.1 + ref.abs() * 2.0 ** -8
            assert bool(((out[t].double() - ref).abs() <= tol).all())
        total = step.lens.tolist()
        keep = [0 if step_no == 4 and b == 1 else n - int(rng.integers(0, min(3, int(a) + 1))) for b, (n, a) in enumerate(zip(total, new))]
        keep = [max(n, 0) for n in keep]
        lens = lib.kv_pages_truncate(step.lens, torch.tensor(keep, dtype=I32, device="cuda"), table, stack, count, page, ws=ws)
        for b, n in enumerate(keep):
            del history[b][n:]
        assert lib.w4a8_device_error(ws) == 0
    lib.kv_pages_truncate(lens, torch.zeros_like(lens), table, stack, count, page, ws=ws)
    assert int(count) == pages and sorted(stack.tolist()) == list(range(pages))
