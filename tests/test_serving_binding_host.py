"""CPU checks of the Python binding of the page maps, the rotation and the 4-bit cache, with stand-ins for tensors on a GPU
and for the library: what is refused is never launched."""
from types import SimpleNamespace

import pytest
import torch

import w4a8_moe_gb300 as pkg

DEVICE = 1
I32, U8, BF16 = torch.int32, torch.uint8, torch.bfloat16
NAMES = ("qk_norm_rope", "kv8_norm_rope_write", "kv_pages_extend", "kv_pages_truncate", "kv4_write", "kv4_read", "kv4_attention")


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
    lib = SimpleNamespace(kv4_attention_workspace_size=lambda *a: 4096)
    for name in NAMES:
        setattr(lib, name, lambda *a, name=name: seen.append((name, a)) or 0)
    monkeypatch.setattr(pkg, "_lib", lib)
    monkeypatch.setattr(pkg, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(pkg, "_current_device", lambda: DEVICE, raising=False)
    monkeypatch.setattr(pkg, "_gpus", 2, raising=False)
    return seen


def arguments(name):
    """-> (positional tensors and values, keyword ones)"""
    x = [gpu(3, h, 64, dtype=BF16) for h in (8, 2, 2)]
    vec = [gpu(3, dtype=I32) for _ in range(4)]
    rope = pkg.RopeTable(gpu(16, dtype=torch.int64), 1.0)
    cache8 = [gpu(6, 2, 16, 64, dtype=U8), gpu(6, 2, 16, 64, dtype=U8), gpu(2), gpu(2)]
    cache4 = [gpu(6, 2, 16, 32, dtype=U8), gpu(6, 2, 16, 32, dtype=U8), gpu(6, 2, 16, 2, dtype=BF16), gpu(6, 2, 16, 2, dtype=BF16)]
    ws = gpu(4096, dtype=U8)
    weights = dict(q_weight=gpu(64, dtype=BF16), k_weight=gpu(64, dtype=BF16))
    if name == "qk_norm_rope":
        return [x[0], x[1], vec[0], rope], dict(weights, q_out=gpu(3, 8, 64, dtype=BF16), k_out=gpu(3, 2, 64, dtype=BF16))
    if name == "kv8_norm_rope_write":
        return [*x, vec[0], vec[1], rope, *cache8], dict(weights, q_out=gpu(3, 8, 64, dtype=BF16))
    pool = [gpu(3, 4, dtype=I32), gpu(6, dtype=I32), gpu(1, dtype=I32), 16]
    if name == "kv_pages_extend":
        out = pkg.PageStep(gpu(4, dtype=I32), *[gpu(9, dtype=I32) for _ in range(4)], gpu(3, dtype=I32))
        return [vec[0], vec[1], *pool, 9], dict(out=out, ws=ws)
    if name == "kv_pages_truncate":
        return [vec[0], vec[1], *pool], dict(out=vec[2], ws=ws)
    if name == "kv4_write":
        return [x[1], x[2], vec[0], *cache4], {}
    if name == "kv4_read":
        return [*cache4, vec[0]], dict(k_out=x[1], v_out=x[2])
    return [x[0], *cache4, gpu(5, 4, dtype=I32), vec[0], vec[1]], dict(out=gpu(3, 8, 64, dtype=BF16), lse=gpu(3, 8), ws=ws)


def every_tensor(args, kw):
    """(what, the arguments with one tensor replaced by what `change` makes of it) for each tensor"""
    def variants(value):
        if isinstance(value, torch.Tensor):
            yield lambda f: f(value)
        elif isinstance(value, tuple):
            for i, v in enumerate(value):
                if isinstance(v, torch.Tensor):
                    yield lambda f, i=i: type(value)(*value[:i], f(value[i]), *value[i + 1:])
    for i, a in enumerate(args):
        for v in variants(a):
            yield i, lambda f, v=v, i=i: ([*args[:i], v(f), *args[i + 1:]], kw)
    for k, a in kw.items():
        for v in variants(a):
            yield k, lambda f, v=v, k=k: (args, dict(kw, **{k: v(f)}))


@pytest.mark.parametrize("name", NAMES)
def test_call_on_the_tensors_gpu_and_stream(calls, name):
    args, kw = arguments(name)
    getattr(pkg, name)(*args, **kw)
    getattr(pkg, name)(*args, **kw, stream=SimpleNamespace(device_index=DEVICE, cuda_stream=77))
    assert [c[0] for c in calls] == [name] * 2
    assert calls[0][1][-1] == 1000 + DEVICE and calls[1][1][-1] == 77


@pytest.mark.parametrize("name", NAMES)
def test_call_is_refused_while_another_gpu_is_current(calls, monkeypatch, name):
    monkeypatch.setattr(pkg, "_current_device", lambda: 0, raising=False)
    args, kw = arguments(name)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        getattr(pkg, name)(*args, **kw)
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_stream_of_another_gpu_is_refused(calls, name):
    args, kw = arguments(name)
    with pytest.raises(ValueError, match="stream"):
        getattr(pkg, name)(*args, **kw, stream=SimpleNamespace(device_index=0, cuda_stream=77))
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_each_tensor_on_another_gpu_or_the_host_is_refused(calls, name):
    args, kw = arguments(name)

    def elsewhere(t):
        t = t.clone().as_subclass(OnGpu)
        t.index = 0
        return t

    for what, change in every_tensor(args, kw):
        for f in (elsewhere, lambda t: torch.zeros(t.shape, dtype=t.dtype)):
            a, k = change(f)
            with pytest.raises(ValueError):
                getattr(pkg, name)(*a, **k)
                pytest.fail(str(what))
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_each_tensor_of_another_type_is_refused(calls, name):
    args, kw = arguments(name)
    for what, change in every_tensor(args, kw):
        if what == "ws":
            continue   # a workspace is bytes of any type
        a, k = change(lambda t: gpu(*t.shape, dtype=torch.float16))
        with pytest.raises(ValueError):
            getattr(pkg, name)(*a, **k)
            pytest.fail(str(what))
    assert not calls


@pytest.mark.parametrize("name", NAMES)
def test_each_tensor_that_repeats_or_skips_its_memory(calls, name):
    """Views whose elements are not where a contiguous tensor has them: refused, but for rows that may lie apart."""
    args, kw = arguments(name)
    for what, change in every_tensor(args, kw):
        def spread(t):
            return gpu(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2].as_subclass(OnGpu)

        a, k = change(spread)
        if any(t.numel() == 1 for t in [*a, *k.values()] if isinstance(t, torch.Tensor) and not t.is_contiguous()):
            continue
        if what == 4 and name == "kv_pages_extend" or what == 4 and name == "kv_pages_truncate":
            continue   # free_count: one element lies nowhere else
        with pytest.raises(ValueError):
            getattr(pkg, name)(*a, **k)
            pytest.fail(str(what))
    assert not calls


def test_rotation_without_keys(calls):
    args, kw = arguments("qk_norm_rope")
    q_out, k_out = pkg.qk_norm_rope(args[0], None, *args[2:], q_out=kw["q_out"])
    got = calls[0][1]
    assert q_out is kw["q_out"] and k_out is None
    assert got[3] is None and got[4] == got[5] == 0 and got[18] is None


def test_attention_table_rows(calls):
    """Without `seqs` every token has a row; with them the table may have any number."""
    args, kw = arguments("kv4_attention")
    with pytest.raises(ValueError, match="row for each token"):
        pkg.kv4_attention(*args[:-1], **kw)
    out, lse = pkg.kv4_attention(*args[:5], gpu(3, 4, dtype=I32), args[6], **dict(kw, lse=False))
    got = calls[0][1]
    assert out is kw["out"] and lse is None and got[14] == 3 and got[15] == 4 and got[16] is None and got[21] is None


def test_workspace_has_to_be_as_large_as_it_says(calls):
    """A view that repeats its memory counts bytes that are not there."""
    for name in ("kv_pages_extend", "kv_pages_truncate", "kv4_attention"):
        args, kw = arguments(name)
        for ws in (gpu(1, dtype=U8).expand(4096), gpu(8192, dtype=U8)[::2]):
            with pytest.raises(ValueError, match="ws"):
                getattr(pkg, name)(*args, **dict(kw, ws=ws.as_subclass(OnGpu)))
    assert not calls


def test_page_tables_whose_rows_share_memory_are_refused_by_the_sizes(calls):
    """An expanded table has a row stride of 0, which the library refuses (a stride below max_pages)."""
    args, kw = arguments("kv_pages_extend")
    args[2] = gpu(1, 4, dtype=I32).expand(3, 4).as_subclass(OnGpu)
    pkg.kv_pages_extend(*args, **kw)
    assert calls[0][1][4] == 0
