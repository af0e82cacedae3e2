"""Decoding with one decoder layer: attention over an FP8 key/value cache whose
first tokens all sequences share, then the W4A8 mixture-of-experts FFN.

A prompt is written into the cache once (kv8_write); every step then projects
the batch's hidden states (fp8_linear), writes their keys and values, attends
over the shared prompt and each sequence's own tokens (kv8_prefix_attention),
projects back, routes and runs the experts (moe_route_gate, moe_w4a8_forward).
At the end one sequence's own tokens are read back (kv8_read), as a program does
that moves a sequence elsewhere. Weights and inputs are random.

    python examples/shared_prefix_decode.py                    # a small layer
    python examples/shared_prefix_decode.py --grok             # Grok-1's shapes, 32 sequences behind 1024 tokens
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a8_moe_gb300 as w4a8  # noqa: E402

SMALL = SimpleNamespace(hidden=512, inter=512, experts=8, top_k=2, heads=12, kv_heads=2, d=128, cap=0.0)
GROK = SimpleNamespace(hidden=6144, inter=32768, experts=8, top_k=2, heads=48, kv_heads=8, d=128, cap=30.0)


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-5)).to(torch.bfloat16)


class Layer:
    """One decoder layer's weights, quantized as the library wants them."""

    def __init__(self, s, gen):
        def rand(*shape):
            return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(0.02).to(torch.bfloat16)

        self.s = s
        self.w_qkv = w4a8.w4a8_quantize_act(rand((s.heads + 2 * s.kv_heads) * s.d, s.hidden))
        self.w_o = w4a8.w4a8_quantize_act(rand(s.hidden, s.heads * s.d))
        self.gate = rand(s.experts, s.hidden)
        self.gate_up = w4a8.w4a8_quantize_experts(rand(s.experts, 2 * s.inter, s.hidden))
        self.down = w4a8.w4a8_quantize_experts(rand(s.experts, s.hidden, s.inter))
        self.a2 = torch.tensor([0.05], device="cuda")

    def qkv(self, x):
        s = self.s
        y = w4a8.fp8_linear(*w4a8.w4a8_quantize_act(norm(x)), *self.w_qkv)
        q, k, v = y.split([s.heads * s.d, s.kv_heads * s.d, s.kv_heads * s.d], 1)   # columns of one tensor: no copies
        return q.unflatten(1, (s.heads, s.d)), k.unflatten(1, (s.kv_heads, s.d)), v.unflatten(1, (s.kv_heads, s.d))

    def ffn(self, x):
        route, _ = w4a8.moe_route_gate(x, self.gate, self.s.top_k)
        xq, a1 = w4a8.w4a8_quantize_act(x)
        return w4a8.moe_w4a8_forward(xq, a1, *self.gate_up, *self.down, self.a2, 0, route)


class Cache:
    """A paged cache with per-token scales; pages [0, n_prefix) hold the prompt, the rest belong to the sequences."""

    def __init__(self, s, prompt, batch, own, page):
        self.page, self.n_prefix = page, -(-prompt // page)
        per = -(-own // page)
        pages = self.n_prefix + batch * per
        self.k, self.v = (torch.zeros(pages, s.kv_heads, page, s.d, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(pages, s.kv_heads, page, device="cuda") for _ in range(2))
        self.prefix_pages = torch.arange(self.n_prefix, dtype=torch.int32, device="cuda")
        self.table = (self.n_prefix + torch.arange(batch * per, dtype=torch.int32, device="cuda")).view(batch, per)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def tensors(self):
        return self.k, self.v, self.ks, self.vs

    def next_slots(self):
        """The slots of one more token of every sequence, which then counts as theirs."""
        at = self.table.gather(1, (self.lens // self.page).long()[:, None])[:, 0]
        slots = at * self.page + self.lens % self.page
        self.lens += 1
        return slots.to(torch.int32)


def decode(s=SMALL, prompt=100, batch=5, steps=20, page=16, seed=0):
    """Runs `steps` decode steps; returns the last step's hidden states and what its attention saw and gave."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer, cache = Layer(s, gen), Cache(s, prompt, batch, steps, page)
    x = torch.randn(prompt, s.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    _, k, v = layer.qkv(x)
    w4a8.kv8_write(k, v, torch.arange(prompt, dtype=torch.int32, device="cuda"), *cache.tensors())

    size = w4a8.kv8_prefix_attention_workspace_size(batch, s.heads, s.kv_heads, s.d, prompt, cache.table.shape[1], page)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    h = torch.randn(batch, s.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(steps):
        if step == min(3, steps - 1):
            start.record()
        q, k, v = layer.qkv(h)
        w4a8.kv8_write(k, v, cache.next_slots(), *cache.tensors())
        a, _ = w4a8.kv8_prefix_attention(q, *cache.tensors(), cache.prefix_pages, prompt, cache.table, cache.lens,
                                         logit_cap=s.cap, ws=ws)
        h = h + w4a8.fp8_linear(*w4a8.w4a8_quantize_act(a.view(batch, -1)), *layer.w_o)
        h = h + layer.ffn(norm(h))
    stop.record()
    # one sequence's own tokens, as keys and values in bf16
    i = torch.arange(steps, device="cuda")
    slots = (cache.table[0][i // page] * page + i % page).to(torch.int32)
    own_k, own_v = w4a8.kv8_read(*cache.tensors(), slots)
    torch.cuda.synchronize()
    assert w4a8.w4a8_device_error(ws) == 0
    ms = start.elapsed_time(stop) / max(1, steps - min(3, steps - 1))
    return SimpleNamespace(hidden=h, q=q, attention=a, cache=cache, own_k=own_k, own_v=own_v, ms_per_step=ms)


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--grok", action="store_true", help="Grok-1's shapes")
    p.add_argument("--prompt", type=int)
    p.add_argument("--batch", type=int)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    r = decode(GROK if a.grok else SMALL, a.prompt or (1024 if a.grok else 100), a.batch or (32 if a.grok else 5), a.steps,
               64 if a.grok else 16)
    print(f"{a.steps} steps, {r.ms_per_step:.3f} ms each; hidden {tuple(r.hidden.shape)}, "
          f"rms {float(r.hidden.float().square().mean().sqrt()):.3f}")
