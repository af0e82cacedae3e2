"""The shared-prefix decoding example: what its attention gave is the softmax
over the keys and values that are read back from its cache."""
import importlib.util
import os

import pytest
import torch

from helpers import ROOT, ensure_built

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,batch,steps", [(100, 5, 20), (700, 40, 3), (16, 1, 1)])
def test_example_decodes(prompt, batch, steps):
    ensure_built()
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "shared_prefix_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.decode(prompt=prompt, batch=batch, steps=steps)
    assert bool(torch.isfinite(r.hidden.float()).all())
    s, c = example.SMALL, r.cache
    assert c.lens.tolist() == [steps] * batch
    i = torch.arange(prompt, device="cuda", dtype=torch.int32)
    pk, pv = example.w4a8.kv8_read(*c.tensors(), i)
    k = torch.cat([pk, r.own_k]).double().transpose(0, 1)   # [kv heads, keys, D] of sequence 0
    v = torch.cat([pv, r.own_v]).double().transpose(0, 1)
    q = r.q[0].double().reshape(s.kv_heads, s.heads // s.kv_heads, s.d)
    x = q @ k.transpose(1, 2) * s.d ** -0.5
    w = torch.softmax(x, -1)
    want, mag = w @ v, w @ v.abs()
    # the keys and values read back carry bf16's rounding (2^-8 of each), the
    # output another; a score's error d moves its weight by 2 d at most twice over
    d = (2.0 ** -8 * (q.abs() @ k.abs().transpose(1, 2)) * s.d ** -0.5).amax(-1, keepdim=True)
    tol = (2.2 * d + 2.0 ** -7) * mag + 2.0 ** -8 * want.abs() + 1e-6
    got = r.attention[0].double().reshape(want.shape)
    assert bool(((got - want).abs() <= tol).all())
