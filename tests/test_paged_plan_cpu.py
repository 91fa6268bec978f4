"""How a shared prefix and the sequences' own keys divide the GPU, asked of the library without a device.

The own keys' lengths are on the device and a captured graph keeps its plan, so the plan must serve them all: what
a table has room for bounds the lengths and says no more."""
import os
import random

import pytest

import exact_attention_30_gb300 as fa
from exact_attention_30_gb300 import build as fa_build

SMS = 152


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(fa.library_path()):
        fa_build.build()
    return fa.load_library()


def _plan(B, hq, hkv, nq, prefix, d, table_keys, page=16, sms=SMS):
    return fa.fa_decode_shared_plan(B, hq, hkv, nq, prefix, d, page, -(-table_keys // page), sms)


@pytest.mark.parametrize("B,hq,prefix,longest", [(32, 32, 4096, 1500), (128, 32, 16384, 1024), (64, 64, 32768, 700)])
def test_wider_tables_leave_the_prefix_its_sms(B, hq, prefix, longest):
    """Conversations, samples and questions, in a table of their longest sequence and in a server's. The prefix alone
    takes most of the time of all three: a plan for long own keys would leave it one range a unit, 8 or 16 SMs."""
    ranges, ctas = _plan(B, hq, 8, 1, prefix, 128, longest)
    assert SMS // 2 <= ctas <= SMS and ctas % ranges == 0
    for keys in (4 * longest, 8192, 32768, 131072, 1 << 30):
        wide = _plan(B, hq, 8, 1, prefix, 128, keys)
        assert abs(wide[0] - ranges) <= 1 and wide[1] >= SMS // 2, (keys, wide, ranges)


def test_tables_beyond_2048_keys_change_nothing():
    rng = random.Random(1)
    for _ in range(300):
        hkv, g, nq = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([1, 1, 2, 3])
        if g * nq > 64:
            continue
        sizes = (rng.randint(1, 400), hkv * g, hkv, nq, rng.randint(0, 60000), rng.choice([64, 128]))
        page = rng.choice([8, 16, 64, 128])
        want = _plan(*sizes, 2048, page)
        for keys in (4096, 20000, 131072):
            assert _plan(*sizes, keys, page) == want, (sizes, page, keys)


def test_plans_fit_their_kernels():
    rng = random.Random(2)
    for _ in range(500):
        hkv, g = rng.choice([1, 2, 3, 8, 32]), rng.choice([1, 2, 4, 8, 33, 64])
        B, prefix, sms = rng.randint(1, 300), rng.randint(0, 40000), rng.choice([1, 20, 148, 152])
        ranges, ctas = _plan(B, hkv * g, hkv, 1, prefix, 128, rng.choice([8, 40, 700, 5000]), 8, sms)
        rows = B * g
        if prefix == 0 or rows <= 32:
            assert (ranges, ctas) == (0, 0)
        else:
            assert 1 <= ranges <= min(64, -(-prefix // 128)) and ctas == -(-rows // 256) * hkv * ranges


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), fa.FA_ERR_INVALID_ARG), (dict(hq=6), fa.FA_ERR_INVALID_ARG), (dict(nq=0), fa.FA_ERR_INVALID_ARG),
    (dict(prefix=-1), fa.FA_ERR_INVALID_ARG), (dict(prefix=(1 << 30) + 1), fa.FA_ERR_INVALID_ARG),
    (dict(table_keys=0), fa.FA_ERR_INVALID_ARG), (dict(sms=-1), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(page=12), fa.FA_ERR_UNSUPPORTED), (dict(hq=64, nq=9), fa.FA_ERR_UNSUPPORTED),
])
def test_plan_refusals(kw, code):
    with pytest.raises(fa.FAError) as e:
        _plan(**{**dict(B=4, hq=8, hkv=4, nq=1, prefix=500, d=128, table_keys=100), **kw})
    assert e.value.code == code


def test_a_gpu_of_too_many_sms_is_refused():
    """The plan counts three CTAs on each SM in 32 bits."""
    ranges, ctas = _plan(40, 8, 4, 1, 5000, 128, 100, sms=65536)  # 80 rows: one block of 256 for each of 4 heads
    assert 1 <= ranges <= 40 and ctas == 4 * ranges
    with pytest.raises(fa.FAError):
        _plan(40, 8, 4, 1, 5000, 128, 100, sms=65537)
    with pytest.raises(fa.FAError):
        _plan(40, 8, 4, 1, 5000, 128, 100, sms=(1 << 31) - 1)


def test_lengths_past_32_bits_are_refused():
    with pytest.raises(ValueError, match="32 bits"):
        _plan(4, 8, 4, 1, (1 << 32) + 500, 128, 100)
    with pytest.raises(ValueError, match="32 bits"):
        fa.fa_decode_shared_workspace_bytes(4, 8, 4, 1, (1 << 32) + 500, 128)
