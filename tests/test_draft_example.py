"""The example that decodes drafted tokens over the 4-bit cache: it runs, its bookkeeping adds up, and its attention is the
dense one over what the cache holds."""
import os
import sys

import pytest
import torch

from helpers import ROOT, ensure_built

pytestmark = pytest.mark.gpu


def test_draft_decode():
    ensure_built()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_decode
    import w4a8_moe_gb300 as w4a8

    steps, drafts, batch, page = 12, 3, 5, 16
    r = draft_decode.decode(batch=batch, drafts=drafts, steps=steps, page=page, seed=3)
    s, c = draft_decode.SMALL, r.cache
    lens = [sum(x) for x in zip(*r.accepted)]
    assert c.lens.tolist() == lens
    used = [-(-n // page) for n in lens]
    assert int(c.count) == c.free.numel() - sum(used)
    held = [p for row, n in zip(c.table.tolist(), used) for p in row[:n]]
    assert sorted(held + c.free.tolist()[:int(c.count)]) == list(range(c.free.numel()))
    # the last step's attention; its rejected drafts' rows are still in the cache, in pages that nobody has taken since
    seqs, seen = r.seqs.tolist(), r.seen.tolist()
    group = s.heads // s.kv_heads
    assert seqs == [b for b in range(batch) for _ in range(drafts)]
    for t in range(0, batch * drafts, 2):
        i = torch.arange(seen[t], device="cuda")
        slots = (c.table[seqs[t]][i // page] * page + i % page).to(torch.int32)
        k, v = (x.double() for x in w4a8.kv4_read(*c.codes, *c.scales, slots))
        q = r.q[t].double().view(s.kv_heads, group, s.d)
        x = torch.einsum("hgd,nhd->hgn", q, k) * s.d ** -0.5
        w = torch.softmax(x, -1)
        want = torch.einsum("hgn,nhd->hgd", w, v).reshape(s.heads, s.d)
        # k and v are read rounded to bf16 (2^-8 of each value), the weights are rounded to f16, the output to bf16
        ds = (torch.einsum("hgd,nhd->hgn", q.abs(), k.abs()) * s.d ** -0.5).amax(-1).reshape(s.heads, 1)
        mag = torch.einsum("hgn,nhd->hgd", w, v.abs()).reshape(s.heads, s.d)
        tol = (2 * ds * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10) * mag * 1.1 + want.abs() * 2.0 ** -8
        got = r.attention[t].double()
        assert bool(((got - want).abs() <= tol).all())
