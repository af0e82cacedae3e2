"""Calls of every kind on one workspace whose header was zeroed once: each leaves the counters there at zero, and none
changes what another computes."""
import pytest
import torch

from helpers import MoECase, ensure_built
from test_kv4 import Batch as Batch4
from test_kv8 import Batch as Batch8

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


@pytest.fixture(scope="module")
def layer():
    ensure_built()
    return MoECase(16, 256, 512, 8, 2, 0, seed=3)


def dynamic(lib, c, ws):
    return lib.moe_w4a8_forward_dynamic(c.xq, c.a1, c.w_gu, c.s_gu, c.w_d, c.s_d, c.act, c.route, ws=ws)


def test_long_attention_after_the_dynamic_forward(lib, layer):
    """Layers of both in turn, with so many keys that the attention shares its work out by counters in the header."""
    b = Batch4([7000 - 13 * i for i in range(40)], 32, 8, 128, 64, seed=71)
    size = max(lib.kv4_attention_workspace_size(40, 32, 8, 128, b.table.shape[1], 64),
               lib.moe_w4a8_dynamic_workspace_size(layer.T, layer.H, layer.I, layer.E, layer.k))
    own, alone = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    want, (y, a2) = b.run(lib, ws=alone), dynamic(lib, layer, alone)
    assert float(a2) != 0
    for _ in range(3):
        got_y, got_a2 = dynamic(lib, layer, own)
        got = b.run(lib, ws=own)
        assert torch.equal(got_y, y) and torch.equal(got_a2, a2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert lib.w4a8_device_error(own) == 0


def test_every_call_leaves_the_header_zero(lib, layer):
    """Small and large calls of all entry points that take a workspace."""
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    c = layer
    vec = torch.randn(16, 256, device="cuda").to(torch.bfloat16)
    gate = torch.randn(8, 256, device="cuda").to(torch.bfloat16)
    codes = torch.randint(0, 120, (256, 256), device="cuda", dtype=torch.uint8)
    one = torch.ones(1, device="cuda")
    kv4 = [Batch4([7000] * 40, 32, 8, 128, 64, seed=72), Batch4([300, 7, 0], 8, 8, 64, 16, seed=73, drafts=3)]
    kv8 = [Batch8([300, 7, 60], 0, 8, 2, 64, 16, 1, seed=74), Batch8([30] * 20, 4000, 48, 8, 128, 64, 0, seed=75)]
    big = MoECase(200, 256, 512, 8, 2, 0, seed=4)
    lens = torch.tensor([5, 0, 33], dtype=I32, device="cuda")
    many = torch.full((700,), 200, dtype=I32, device="cuda")

    def pages(n, add):
        b = n.numel()
        table = torch.arange(b * 40, dtype=I32, device="cuda").view(b, 40)
        stack, count = torch.arange(b * 40, dtype=I32, device="cuda"), torch.tensor([b * 20], dtype=I32, device="cuda")
        step = lib.kv_pages_extend(n, torch.full_like(n, add), table, stack, count, 16, b * add, ws=ws)
        lib.kv_pages_truncate(step.lens, n, table, stack, count, 16, ws=ws)

    calls = {
        "quantize": lambda: lib.w4a8_quantize_act(vec, ws=ws),
        "route": lambda: lib.moe_route(c.inp["logits"], 2, ws=ws),
        "route and gate": lambda: lib.moe_route_gate(vec, gate, 2, ws=ws),
        "forward": lambda: lib.moe_w4a8_forward(c.xq, c.a1, c.w_gu, c.s_gu, c.w_d, c.s_d, c.a2, c.act, c.route, ws=ws),
        "larger forward": lambda: big.run_gpu(ws=ws),
        "dynamic": lambda: dynamic(lib, c, ws),
        "larger dynamic": lambda: dynamic(lib, big, ws),
        "block linear": lambda: lib.fp8_block_linear(vec, codes, torch.ones(2, 2, device="cuda"), ws=ws),
        "linear": lambda: lib.fp8_linear(codes, one, codes, one, ws=ws),
        "pages": lambda: pages(lens, 3),
        "many pages": lambda: pages(many, 200),
        "4 bits, long": lambda: kv4[0].run(lib, ws=ws),
        "4 bits, several tokens": lambda: kv4[1].run(lib, ws=ws),
        "FP8": lambda: kv8[0].run(lib, ws=ws),
        "FP8 over a prefix": lambda: kv8[1].run(lib, ws=ws),
    }
    for what, call in calls.items():
        ws[256:].zero_()   # (the linear layer wants its counters, behind the header, zero before its first call)
        call()
        assert bool((ws[:256] == 0).all()), what
