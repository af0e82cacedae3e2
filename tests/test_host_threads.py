"""Calls from several host threads at once whose kernels need different amounts of shared memory: every one of them is
launched, and gives what it gives alone."""
import subprocess
import sys
import threading

import pytest
import torch

from helpers import ROOT, ensure_built
from test_kv4 import Batch as Batch4
from test_kv8 import Batch as Batch8

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg


class Recorder:
    """The library, with the arguments of every call that went to it."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        f = getattr(self.real, name)

        def call(*args):
            self.calls.append((f, args))
            return f(*args)
        return call


def at_once(lib, monkeypatch, calls, outputs, times=1500):
    """Makes each of `calls` on a stream of its own, then all of them again and again from a thread each, straight through
    the C entry points; what they wrote has to be what they wrote alone."""
    recorder = Recorder(lib._load())
    monkeypatch.setattr(lib, "_lib", recorder)
    made = []
    for call in calls:
        recorder.calls = []
        call(torch.cuda.Stream())
        made.append([c for c in recorder.calls if c[1] and not c[0].__name__.endswith("size")])
    monkeypatch.undo()
    torch.cuda.synchronize()
    want = [x.clone() for x in outputs]
    refused, gate = [], threading.Barrier(len(made))

    def work(own):
        gate.wait()
        for _ in range(times):
            refused.extend(s for s in [f(*args) for f, args in own] if s)

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(own,)) for own in made]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[0])
    assert all(torch.equal(x, y) for x, y in zip(outputs, want))


@pytest.mark.parametrize("hq,hkv,drafts", [(1, 1, 1), (1, 1, 4), (16, 1, 1)])
def test_attention_over_4_bits(lib, monkeypatch, hq, hkv, drafts):
    calls, outputs = [], []
    for tokens in (4096, 2000, 4096, 3000):
        b = Batch4([i % 5 for i in range(tokens // drafts)], hq, hkv, 128, 16, seed=81, drafts=drafts)
        ws = torch.zeros(lib.kv4_attention_workspace_size(tokens, hq, hkv, 128, 1, 16), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(b.q), torch.empty(tokens, hq, device="cuda")
        calls.append(lambda s, b=b, ws=ws, out=out, lse=lse: b.run(lib, ws=ws, out=out, lse=lse, stream=s))
        outputs += [out, lse]
    at_once(lib, monkeypatch, calls, outputs)


@pytest.mark.parametrize("hq,hkv,mode", [(1, 1, 0), (16, 1, 1)])
def test_attention_over_8_bits(lib, monkeypatch, hq, hkv, mode):
    calls, outputs = [], []
    for batch in (4096, 2900, 4096, 3500):
        b = Batch8([i % 5 for i in range(batch)], 0, hq, hkv, 128, 16, mode, seed=82)
        ws = torch.zeros(lib.kv8_prefix_attention_workspace_size(batch, hq, hkv, 128, 0, 10, 16), dtype=torch.uint8,
                         device="cuda")
        out, lse = torch.empty_like(b.q), torch.empty(batch, hq, device="cuda")
        calls.append(lambda s, b=b, ws=ws, out=out, lse=lse: b.run(lib, ws=ws, out=out, lse=lse, stream=s))
        outputs += [out, lse]
    at_once(lib, monkeypatch, calls, outputs)


def test_page_tables(lib, monkeypatch):
    """No pages move (all tokens fit their last page), so that every call finds what the first one found."""
    calls, outputs = [], []
    for batch in (4096, 4050, 4096, 4020):
        lens = torch.tensor([1 + b % 13 for b in range(batch)], dtype=I32, device="cuda")
        new = torch.tensor([b % 3 for b in range(batch)], dtype=I32, device="cuda")
        pool = (torch.arange(batch, dtype=I32, device="cuda").view(batch, 1), torch.arange(batch, dtype=I32, device="cuda"),
                torch.zeros(1, dtype=I32, device="cuda"), 16)
        ws = torch.zeros(lib.kv_pages_workspace_size(), dtype=torch.uint8, device="cuda")
        step = lib.PageStep(*[torch.empty(n, dtype=I32, device="cuda") for n in [batch + 1] + [2 * batch] * 4 + [batch]])
        calls.append(lambda s, a=(lens, new, *pool), step=step, ws=ws, batch=batch:
                     lib.kv_pages_extend(*a, 2 * batch, out=step, ws=ws, stream=s))
        outputs += step
    at_once(lib, monkeypatch, calls, outputs)


CHILD = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import w4a8_moe_gb300 as lib
from test_kv8 import Batch
for batch in range(2678, 2692):
    b = Batch([i % 5 for i in range(batch)], 0, {hq}, 1, 128, 16, {mode}, seed=batch)
    b.check(*b.run(lib), every=211)
print("all right")
"""


@pytest.mark.parametrize("hq,mode", [(1, 0), (1, 1), (16, 0), (16, 1)])
def test_attention_over_8_bits_at_the_shared_memory_that_needs_no_asking(lib, hq, mode):
    """In a process of its own: a larger batch before would have asked for more already."""
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, hq=hq, mode=mode)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "all right" in r.stdout, r.stderr[-2000:]
