"""Giving pages back where a row of the table holds a number that is no page: that sequence stays as it is, and no such number
comes to the stack."""
import numpy as np
import pytest
import torch

from helpers import ensure_built
from test_pages import Pool, W4A8_ERR_INDEX, ceil, same_pool, workspace

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


@pytest.mark.parametrize("batch,page,longest,broken", [
    (1, 16, 100, 1), (5, 16, 70, 2), (40, 64, 5000, 1), (300, 256, 2000, 17), (1000, 16, 400, 1), (4096, 16, 33, 40),
    (3, 16, 100000, 1),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_truncate_leaves_broken_sequences(lib, batch, page, longest, broken, in_place):
    rng = np.random.default_rng(batch)
    lens = rng.integers(longest // 2, longest + 1, batch).tolist()
    p = Pool(lens, page, ceil(longest, page) + 2, spare=3, seed=batch)
    state = p.gpu()
    table = state[1]
    keep = [0 if rng.random() < 0.3 else int(rng.integers(0, n + 1)) for n in lens]
    picked = rng.permutation(batch)[:broken].tolist()
    for i, b in enumerate(picked):
        keep[b] = min(keep[b], (len(p.rows[b]) - 1) * page)   # a page of it at least would go
        at = int(rng.integers(ceil(keep[b], page), len(p.rows[b])))
        for where in (table, torch.from_numpy(p.stale)):
            where[b, at] = [p.num, -1, 2 ** 31 - 1, -2 ** 31][i % 4]
        if keep[b] >= page:   # a second one, in the part that stays
            table[b, 0] = p.stale[b, 0] = -5
    others = [b for b in range(batch) if b not in picked and keep[b] >= page]
    if others:   # one that is broken only where nothing goes back is given back as any other
        table[others[0], 0] = p.stale[others[0], 0] = p.num + 7
        p.rows[others[0]][0] = p.num + 7
    ws = workspace(lib)
    want = [n if b in picked else k for b, (n, k) in enumerate(zip(lens, keep))]
    for again in range(2):   # the second time only the broken ones are left to give, and stay again
        after = lib.kv_pages_truncate(state[0], torch.tensor(keep, dtype=I32, device="cuda"), *state[1:], page,
                                      out=state[0] if in_place else None, ws=ws)
        p.truncate(want)
        same_pool(p, *state[1:], after)
        assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX
        assert bool((ws == 0).all())
        state = (after, *state[1:])
    # mended, they go back too
    for b in picked:
        row = torch.tensor(p.rows[b], dtype=I32)
        table[b, :len(row)] = row.cuda()
        p.stale[b, :len(row)] = row.numpy()
    after = lib.kv_pages_truncate(state[0], torch.tensor(keep, dtype=I32, device="cuda"), *state[1:], page, ws=ws)
    p.truncate(keep)
    same_pool(p, *state[1:], after)
    assert lib.w4a8_device_error(ws) == 0


def test_a_broken_row_beside_lengths_out_of_range_and_a_full_stack(lib):
    ws = workspace(lib)
    p = Pool([100, 64, 40, 50], 16, 8, spare=0)
    lens, table, stack, count = p.gpu()
    table[1, 3] = -2
    before = stack.clone()
    keep = torch.tensor([101, 20, 10, -1], dtype=I32, device="cuda")   # only the third can go
    got = lib.kv_pages_truncate(lens, keep, table, stack, count, 16, ws=ws)
    assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX and got.tolist() == [100, 64, 10, 50]
    assert int(count) == 2 and stack[:2].tolist() == [int(table[2, 2]), int(table[2, 1])]
    assert torch.equal(stack[4:], before[4:])   # (what four pages would have taken is written to)
    # a count that leaves room for what the whole ones give, but not for the broken ones' too: the whole ones go
    count.fill_(p.num - 2)
    keep = torch.tensor([100, 0, 10, 50], dtype=I32, device="cuda")
    got = lib.kv_pages_truncate(lens, keep, table, stack, count, 16, ws=ws)
    assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX and got.tolist() == [100, 64, 10, 50] and int(count) == p.num
    # and one that leaves no room for those either: nothing goes
    count.fill_(p.num - 1)
    before = stack.clone()
    got = lib.kv_pages_truncate(lens, keep, table, stack, count, 16, ws=ws)
    assert lib.w4a8_device_error(ws) == W4A8_ERR_INDEX and torch.equal(got, lens)
    assert int(count) == p.num - 1 and torch.equal(stack, before)
