"""Rows of weights that lie upon one another are refused by every entry point that writes them, and no others are."""
import itertools

import numpy as np
import pytest

import test_prompt_cpu
from test_prompt_cpu import FAKE, INVALID, _cache, _evict, _step, _weights, _weights_paged, lib  # noqa: F401


def _overlap(b, h, keys, sb, sh):
    """Whether any two of the b * h rows share an element."""
    at = np.sort((np.arange(b)[:, None] * sb + np.arange(h)[None] * sh).ravel())
    return bool((np.diff(at) < keys).any())


@pytest.mark.parametrize("b,h", [(1, 1), (1, 3), (3, 1), (2, 2), (2, 3), (3, 2), (5, 4), (4, 7)])
def test_every_pair_of_strides(lib, b, h):
    keys, some = 3, 0
    for sb, sh in itertools.product(range(0, 30), range(0, 30)):
        bad = _overlap(b, h, keys, sb, sh)
        some += bad
        kw = dict(wb=sb, wh=sh, wk=keys, B=b)
        cache = _cache(kv_heads=h)
        got = [_weights(lib, Hq=4 * h, Hkv=h, qs=512 * h, ks=128 * h, **kw),
               _weights_paged(lib, cache, Hq=4 * h, qs=512 * h, **kw), _step(lib, cache, Hq=4 * h, **kw),
               _evict(lib, cache, nw=FAKE + 4096, nwb=4000, nwh=400, **kw),
               _evict(lib, cache, nw=FAKE + 4096, wb=4000, wh=400, wk=keys, B=b, nwb=sb, nwh=sh, budget=3, recent=1)]
        # (without a device what is not refused ends in a CUDA error)
        assert [x == INVALID for x in got] == [bad] * 5, (sb, sh, got)
    assert some > 0 or b == h == 1


def test_far_apart(lib):
    """Strides near the largest ones: no product past 64 bits."""
    for sb, sh in ((1 << 40, 1 << 39), (1 << 20, 1 << 40), (1 << 40, 1 << 40)):
        assert (_weights(lib, wb=sb, wh=sh, wk=200) == INVALID) == (sb == sh)
    for s in ((1 << 40) + 1, 1 << 62, -(1 << 62)):
        assert _weights(lib, wb=s, wh=200, wk=200) == INVALID
        assert _weights(lib, wb=400, wh=s, wk=200) == INVALID
    many = dict(B=65535, kept=FAKE, nw=FAKE + 4096, nwb=1 << 20, nwh=64)
    assert _evict(lib, _cache(kv_heads=1), wb=64, wh=0, **many) != INVALID
    assert _evict(lib, _cache(kv_heads=3), wb=64, wh=65535 * 64 - 1, **many) == INVALID


def test_weights_in_place_keep_their_strides(lib):
    same = dict(nw=FAKE, wk=64, budget=64, recent=8)
    assert _evict(lib, wb=128, wh=64, nwb=128, nwh=64, **same) != INVALID
    for nwb, nwh in ((192, 64), (256, 128), (64, 128)):
        assert _evict(lib, wb=128, wh=64, nwb=nwb, nwh=nwh, **same) == INVALID
        assert _evict(lib, wb=128, wh=64, nwb=nwb, nwh=nwh, **{**same, "nw": FAKE + 4096}) != INVALID
    # an axis of one entry has no stride
    assert _evict(lib, _cache(kv_heads=1), wb=128, wh=1, nwb=128, nwh=99, **same) != INVALID
    assert _evict(lib, wb=1, wh=64, nwb=99, nwh=64, B=1, **same) != INVALID


def test_evict_refusals_with_weights_elsewhere(lib):
    """Each of the other refusals by itself: the call is in order but for it."""
    assert _evict(lib, nw=FAKE + 4096) != INVALID
    for kw, code in test_prompt_cpu.test_evict_refusals.pytestmark[0].args[1]:
        assert _evict(lib, **{"nw": FAKE + 4096, **kw}) == code, kw


def test_tables_in_place_keep_their_width(lib):
    """[B, pages] rows of another width would be other sequences' pages."""
    far = dict(nw=FAKE + 4096)
    assert _evict(lib, max_pages=5, new_pages=4, **far) == INVALID
    assert _evict(lib, max_pages=4, new_pages=5, **far) == INVALID
    assert _evict(lib, max_pages=5, new_pages=4, new=FAKE + 4096, **far) != INVALID
    assert _evict(lib, max_pages=5, new_pages=4, B=1, **far) != INVALID
