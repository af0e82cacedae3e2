"""CPU checks of how the attention over the FP8 cache cuts up a shared prefix."""
import ctypes

import pytest

from helpers import ensure_built


@pytest.fixture(scope="module")
def plan():
    ensure_built()
    import w4a8_moe_gb300 as pkg
    return pkg.kv8_prefix_attention_plan


def test_plan_refusals(plan):
    import w4a8_moe_gb300 as pkg
    lib = pkg._load()
    out = (ctypes.c_int32 * 6)()
    good = [32, 48, 8, 128, 1024, 8, 64, 0, 0.0, 152]
    assert lib.kv8_prefix_attention_plan(*good, None) == 1
    assert lib.kv8_prefix_attention_plan(*good, out) == 0
    for i, bad in ((0, 0), (1, 47), (2, 0), (3, 96), (4, -1), (5, -1), (6, 48), (7, 2), (8, -1.0), (8, float("nan")), (9, 0)):
        assert lib.kv8_prefix_attention_plan(*good[:i], bad, *good[i + 1:], out) == 2, (i, bad)


def test_plan_launches(plan):
    assert plan(32, 48, 8, 128, 8192, 8, 64, num_sms=152)["launches"] == 3
    assert plan(32, 48, 8, 128, 8192, 0, 64, num_sms=152)["launches"] == 2    # no own tokens
    short = plan(1, 48, 8, 128, 1024, 8, 64, num_sms=152)
    assert (short["ranges"], short["tiles_per_range"], short["prefix_blocks"], short["launches"]) == (0, 0, 0, 2)
    assert plan(1, 48, 8, 128, 0, 8, 64, num_sms=152)["launches"] == 2
    assert plan(1, 48, 8, 128, 0, 0, 64, num_sms=152)["launches"] == 1


@pytest.mark.parametrize("num_sms", [100, 132, 148, 152])
def test_plan_fills_the_sms_that_there_are(plan, num_sms):
    """A long prefix is cut so that the waves of blocks are full, on this GPU's number of SMs: no further range or two
    would have had room in the same number of waves."""
    for batch, hq, hkv in ((32, 48, 8), (17, 16, 1), (100, 32, 8), (64, 40, 8), (40, 28, 4)):
        p = plan(batch, hq, hkv, 128, 200000, 0, 64, num_sms=num_sms)
        pairs = hkv * -(-batch * (hq // hkv) // 256)
        assert p["prefix_blocks"] == p["ranges"] * pairs
        waves = -(-p["prefix_blocks"] // num_sms)
        most = min(64, 2 * -(-152 // pairs))
        assert p["prefix_blocks"] + 2 * pairs > waves * num_sms or p["ranges"] >= most - 1, (batch, hq, hkv, p)


@pytest.mark.parametrize("batch,hq,hkv,d,prefix,page,own,scale_mode,cap", [
    (64, 32, 8, 128, 8192, 64, 512, 1, 0.0),
    (128, 48, 8, 128, 32768, 64, 1024, 0, 0.0),
    (256, 48, 8, 128, 65536, 128, 256, 0, 0.0),
    (32, 48, 8, 128, 1024, 64, 256, 0, 30.0),
    (17, 16, 1, 64, 4999, 16, 784, 0, 0.0),
    (24, 32, 8, 128, 3000, 64, 128, 0, 0.0),
    (8, 32, 8, 128, 20000, 64, 128, 0, 0.0),
])
def test_plan_hardly_follows_the_tables_width(plan, batch, hq, hkv, d, prefix, page, own, scale_mode, cap):
    """A page table is as wide as the longest context a program allows, which says little about the lengths: the prefix
    keeps its SMs however wide the table is."""
    tight = plan(batch, hq, hkv, d, prefix, -(-own // page), page, scale_mode, cap, num_sms=152)
    for tokens in (4096, 32768, 131072, 1 << 20):
        wide = plan(batch, hq, hkv, d, prefix, tokens // page, page, scale_mode, cap, num_sms=152)
        assert wide["tiles_per_range"] <= 2 * tight["tiles_per_range"], (tokens, tight, wide)


HEADS = [(48, 8, 128), (32, 8, 128), (28, 4, 128), (8, 1, 128), (16, 1, 128), (16, 1, 64), (64, 8, 64), (8, 8, 128)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("prefix", [0, 5000, 20000])
def test_plan_join_fits_the_sms(plan, hq, hkv, d, prefix):
    """Several warps a row only while the blocks of all rows are on the SMs at once, whatever the tables would allow."""
    for batch in list(range(1, 160)) + [200, 256, 600]:
        for tokens in (64, 1024, 32768, 131072):
            w = plan(batch, hq, hkv, d, prefix, tokens // 64, 64, num_sms=152)["join_warps"]
            fits = {8: 2, 4: 4 if d == 128 else 7, 2: 8}
            assert w in (0, 1) or batch * hq <= fits[w] * 152, (batch, tokens, w)


def test_plan_blocks_of_few_sequences(plan):
    """The form of 16 rows whose registers spill is for very many keys of many sequences, not for wide tables alone."""
    for batch in (1, 17, 40, 64):
        for tokens in (64, 8192, 131072):
            assert plan(batch, 16, 1, 128, 0, tokens // 64, 64, num_sms=152)["own_blocks_per_sm"] == 2
    assert plan(256, 16, 1, 128, 0, 128, 64, num_sms=152)["own_blocks_per_sm"] == 3
    assert plan(256, 16, 1, 64, 0, 1, 64, num_sms=152)["own_blocks_per_sm"] == 3   # D 64 does not spill
