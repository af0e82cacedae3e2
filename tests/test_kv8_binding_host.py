"""CPU checks of the FP8 key/value cache's Python binding, with stand-ins for
tensors on a GPU and for the library: what is refused is never launched."""
from types import SimpleNamespace

import pytest
import torch

import w4a8_moe_gb300 as pkg

DEVICE = 1


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    index = DEVICE

    def get_device(self):
        return self.index

    @property
    def is_cuda(self):
        return True


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library: (name, arguments)."""
    seen = []
    lib = SimpleNamespace(kv8_prefix_attention_workspace_size=lambda *a: 4096)
    for name in ("kv8_write", "kv8_read", "kv8_prefix_attention"):
        setattr(lib, name, lambda *a, name=name: seen.append((name, a)) or 0)
    monkeypatch.setattr(pkg, "_lib", lib)
    monkeypatch.setattr(pkg, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(pkg, "_current_device", lambda: DEVICE, raising=False)
    monkeypatch.setattr(pkg, "_gpus", 2, raising=False)
    return seen


def arguments():
    i32, bf16 = torch.int32, torch.bfloat16
    cache = [gpu(6, 2, 16, 64, dtype=torch.uint8), gpu(6, 2, 16, 64, dtype=torch.uint8), gpu(2), gpu(2)]
    x = [gpu(3, 2, 64, dtype=bf16), gpu(3, 2, 64, dtype=bf16)]
    slots = gpu(3, dtype=i32)
    return {
        "kv8_write": (pkg.kv8_write, (*x, slots, *cache), {}),
        "kv8_read": (pkg.kv8_read, (*cache, slots), dict(k_out=x[0], v_out=x[1])),
        "kv8_prefix_attention": (pkg.kv8_prefix_attention,
                                 (gpu(3, 8, 64, dtype=bf16), *cache, gpu(2, dtype=i32), 20, gpu(3, 4, dtype=i32),
                                  gpu(3, dtype=i32)),
                                 dict(out=gpu(3, 8, 64, dtype=bf16), ws=gpu(4096, dtype=torch.uint8))),
    }


NAMES = ("kv8_write", "kv8_read", "kv8_prefix_attention")


@pytest.mark.parametrize("name", NAMES)
def test_call_on_the_tensors_gpu_and_stream(calls, name):
    fn, args, kw = arguments()[name]
    fn(*args, **kw)
    fn(*args, **kw, stream=SimpleNamespace(device_index=DEVICE, cuda_stream=77))
    assert [c[0] for c in calls] == [name] * 2
    assert calls[0][1][-1] == 1000 + DEVICE and calls[1][1][-1] == 77


@pytest.mark.parametrize("name", NAMES)
def test_call_is_refused_while_another_gpu_is_current(calls, monkeypatch, name):
    """The library launches on the current GPU: with the tensors on another one it must not be called."""
    monkeypatch.setattr(pkg, "_current_device", lambda: 0, raising=False)
    fn, args, kw = arguments()[name]
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        fn(*args, **kw)
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_stream_of_another_gpu_is_refused(calls, name):
    fn, args, kw = arguments()[name]
    with pytest.raises(ValueError, match="stream"):
        fn(*args, **kw, stream=SimpleNamespace(device_index=0, cuda_stream=77))
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_two_gpus_are_refused(calls, name):
    fn, args, kw = arguments()[name]
    for i, x in enumerate(args):
        if isinstance(x, torch.Tensor):
            other = x.clone().as_subclass(OnGpu)
            other.index = 0
            with pytest.raises(ValueError):
                fn(*args[:i], other, *args[i + 1:], **kw)
    assert not calls


def test_attention_without_own_tokens(calls):
    """No page table and no lengths, as in the C call: the prefix alone. `lse=False` asks for none."""
    fn, args, kw = arguments()["kv8_prefix_attention"]
    out, lse = fn(*args[:7], None, None, lse=False, **kw)
    got = calls[0][1]
    assert out is kw["out"] and lse is None
    table, stride, most, lens = got[15:19]
    assert table is None and stride == most == 0 and lens is None
    assert got[22] is None   # lse


def test_attention_refuses_what_is_missing(calls):
    fn, args, kw = arguments()["kv8_prefix_attention"]
    for i, what in ((5, "prefix_pages"), (7, "page_table"), (8, "suffix_lens")):
        with pytest.raises(ValueError, match=what):
            fn(*args[:i], None, *args[i + 1:], **kw)
    assert not calls
    fn(*args[:5], None, 0, *args[7:], **kw)   # no prefix: no pages of it
    assert calls[0][1][13] is None and calls[0][1][14] == 0


def test_workspace_has_to_be_as_large_as_it_says(calls):
    """A view that repeats its memory counts bytes that are not there."""
    fn, args, kw = arguments()["kv8_prefix_attention"]
    for ws in (gpu(1, dtype=torch.uint8).expand(4096), gpu(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws"):
            fn(*args, **dict(kw, ws=ws.as_subclass(OnGpu)))
    assert not calls
