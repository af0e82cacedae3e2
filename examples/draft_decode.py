"""Decoding with drafted tokens over a key/value cache of 4 bits, with one decoder layer whose page tables live on the GPU.

Every step takes a few drafted tokens of each sequence (here random hidden states). Their pages and slots come from the
sequences' lengths (kv_pages_extend); the layer projects them (fp8_linear), norms and rotates queries and keys
(qk_norm_rope), writes keys and values (kv4_write) and attends, each draft to what is before it (kv4_attention), and runs
the experts (moe_route_gate, moe_w4a8_forward). Then the sequences keep as many drafts as were accepted (here a random
number) and give the pages behind them back (kv_pages_truncate). Nothing but the sizes is known on the host, so the step
is captured once and replayed.

    python examples/draft_decode.py                    # a small layer
    python examples/draft_decode.py --drafts 5 --batch 16
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import w4a8_moe_gb300 as w4a8  # noqa: E402
from shared_prefix_decode import Layer, SMALL, norm  # noqa: E402


class Pages:
    """A 4-bit cache and the tables of its pages, all on the GPU."""

    def __init__(self, s, batch, most, page):
        pages = batch * -(-most // page)
        self.page = page
        self.codes = [torch.zeros(pages, s.kv_heads, page, s.d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(pages, s.kv_heads, page, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.table = torch.full((batch, pages // batch), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.free = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.count = torch.tensor([pages], dtype=torch.int32, device="cuda")

    def pool(self):
        return self.table, self.free, self.count, self.page


def decode(s=SMALL, batch=6, drafts=4, steps=20, page=16, seed=0):
    """Runs `steps` steps; returns the pages, the drafts kept of each step and the last step's tensors."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer, cache = Layer(s, gen), Pages(s, batch, steps * drafts, page)
    rope = w4a8.rope_table(s.d, base=500000.0)
    q_norm, k_norm = ((1 + 0.1 * torch.randn(s.d, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))
    tokens = batch * drafts
    new = torch.full((batch,), drafts, dtype=torch.int32, device="cuda")
    kept = torch.zeros(batch, dtype=torch.int32, device="cuda")
    x = torch.zeros(tokens, s.hidden, dtype=torch.bfloat16, device="cuda")
    size = w4a8.kv4_attention_workspace_size(tokens, s.heads, s.kv_heads, s.d, cache.table.shape[1], page)
    ws, pages_ws = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (size, w4a8.kv_pages_workspace_size()))
    last = SimpleNamespace()

    def step():
        at = w4a8.kv_pages_extend(cache.lens, new, *cache.pool(), tokens, ws=pages_ws)
        q, k, v = layer.qkv(x)
        q, k = w4a8.qk_norm_rope(q, k, at.positions, rope, q_norm, k_norm)
        w4a8.kv4_write(k, v, at.slots, *cache.codes, *cache.scales)
        a, _ = w4a8.kv4_attention(q, *cache.codes, *cache.scales, cache.table, at.seen, seqs=at.seqs, logit_cap=s.cap, ws=ws)
        h = x + w4a8.fp8_linear(*w4a8.w4a8_quantize_act(a.view(tokens, -1)), *layer.w_o)
        h = h + layer.ffn(norm(h))
        w4a8.kv_pages_truncate(at.lens, cache.lens + kept, *cache.pool(), out=cache.lens, ws=pages_ws)
        last.q, last.attention, last.hidden, last.seen, last.seqs = q, a, h, at.seen, at.seqs

    def inputs():
        x.copy_(torch.randn(tokens, s.hidden, generator=gen, device="cuda"))
        kept.copy_(torch.randint(0, drafts + 1, (batch,), generator=gen, device="cuda"))
        return kept.tolist()

    accepted = [inputs()]
    side = torch.cuda.Stream()   # the first step outside the graph, as what it sets up cannot be captured
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps - 1):
        accepted.append(inputs())
        graph.replay()
    torch.cuda.synchronize()
    assert w4a8.w4a8_device_error(ws) == 0 and w4a8.w4a8_device_error(pages_ws) == 0
    return SimpleNamespace(cache=cache, accepted=accepted, graph=graph, **vars(last))


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--batch", type=int, default=6)
    p.add_argument("--drafts", type=int, default=4)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    r = decode(batch=a.batch, drafts=a.drafts, steps=a.steps)
    print(f"{a.steps} steps of {a.drafts} drafts; lengths now {r.cache.lens.tolist()}, free pages {int(r.cache.count)}, "
          f"rms {float(r.hidden.float().square().mean().sqrt()):.3f}")
