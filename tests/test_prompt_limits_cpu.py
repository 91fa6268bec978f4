"""The limit of the forward's blocks, as the header names it, and before any CUDA call."""
import pytest

from test_prompt_cpu import INVALID, UNSUPPORTED, _cache, _fwd, _paged, lib  # noqa: F401


def _within(b, t, mq, hq, hkv):
    tokens = 2 * (128 // (hq // hkv))
    return 256 * hkv * min(t // tokens + b, b * -(-mq // tokens)) < 1 << 31


@pytest.mark.parametrize("b,t,mq,hq,hkv", [(1 << 23, 1 << 23, 1, 1, 1), ((1 << 23) - 1, 1 << 23, 1, 4, 1),
                                           (1 << 21, 1 << 21, 1, 4, 4), ((1 << 21) - 1, 1 << 21, 1, 8, 4),
                                           (1 << 12, 1 << 28, 1 << 20, 71, 1), (1 << 12, 1 << 23, 1 << 20, 71, 1),
                                           (1 << 12, (1 << 24) - (1 << 13) - 2, 1 << 23, 128, 1),
                                           (1 << 12, (1 << 24) - (1 << 13), 1 << 23, 128, 1)])
def test_rows_of_all_blocks(lib, b, t, mq, hq, hkv):
    sizes = dict(B=b, t=t, mq=mq, Hq=hq, qs=hq * 128, os_=hq * 128)
    # what is within the limit is refused for its missing keys or tables, which are looked at afterwards
    got = [_fwd(lib, Hkv=hkv, ks=hkv * 128, vs=hkv * 128, tk=t, K=0, **sizes),
           _paged(lib, _cache(kv_heads=hkv), tables=0, **sizes)]
    assert got == [INVALID if _within(b, t, mq, hq, hkv) else UNSUPPORTED] * 2


def test_both_sides_are_tested():
    cases = test_rows_of_all_blocks.pytestmark[0].args[1]
    assert {_within(*c) for c in cases} == {True, False}
