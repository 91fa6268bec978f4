"""Rows of weights that lie upon one another are refused by every entry point that writes them, and no others are."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

import test_prompt_cpu
from exact_attention_30_gb300 import build as fa_build
from test_prompt_cpu import FAKE, INVALID, _cache, _evict, _step, _weights, _weights_paged, lib  # noqa: F401


@pytest.fixture(scope="module")
def rows_ok(tmp_path_factory):
    """The library's check by itself: what it lets through is not launched."""
    d = tmp_path_factory.mktemp("rows")
    csrc = os.path.join(os.path.dirname(fa_build.__file__), "csrc")
    src = d / "rows.cc"
    src.write_text('#include "fa_checks.h"\n'
                   'extern "C" int rows_ok(long long b, long long h, int keys, int B, int H) {\n'
                   "  return fa::weight_strides_ok(b, h, keys, B, H);\n}\n")
    out = str(d / "rows.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(fa_build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", f"-I{csrc}", f"-I{cuda}", str(src), "-o", out], check=True)
    fn = ctypes.CDLL(out).rows_ok
    fn.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    return fn


def _overlap(b, h, keys, sb, sh):
    """Whether any two of the b * h rows share an element."""
    at = np.sort((np.arange(b)[:, None] * sb + np.arange(h)[None] * sh).ravel())
    return bool((np.diff(at) < keys).any())


@pytest.mark.parametrize("b,h", [(1, 1), (1, 3), (3, 1), (2, 2), (2, 3), (3, 2), (5, 4), (4, 7), (9, 30)])
def test_every_pair_of_strides(rows_ok, b, h):
    for keys in (1, 3):
        for sb, sh in itertools.product(range(-3, 40), range(-3, 40)):
            bad = _overlap(b, h, keys, sb, sh) or (b > 1 and sb < 1) or (h > 1 and sh < 1)
            assert bool(rows_ok(sb, sh, keys, b, h)) != bad, (keys, sb, sh)


def test_far_apart(rows_ok):
    """Strides near the largest ones: no product past 64 bits."""
    top = 1 << 40
    for sb, sh, good in ((1 << 20, top, True), (top, 1 << 20, True), (top, top >> 1, False), (top, top, False),
                         (top - 199, top, False), (top - 200, top, True)):  # rows 200 apart just fit
        assert bool(rows_ok(sb, sh, 200, 4096, 4096)) == good, (sb, sh)
    for s in (top + 1, 1 << 62, -(1 << 62)):
        assert not rows_ok(s, 200, 200, 2, 2) and not rows_ok(400, s, 200, 2, 2)
    assert rows_ok(64, 65535 * 64, 64, 65535, 3) and not rows_ok(64, 65535 * 64 - 1, 64, 65535, 3)


@pytest.mark.parametrize("sb,sh", [(200, 200), (400, 399), (399, 200), (200, 399), (0, 200), (200, 0), (-400, 200), (350, 200)])
def test_entry_points_refuse_them(lib, sb, sh):
    kw = dict(wb=sb, wh=sh, wk=200)
    assert _weights(lib, **kw) == INVALID
    assert _weights_paged(lib, **kw) == INVALID
    assert _step(lib, **kw) == INVALID
    far = dict(nw=FAKE + 4096, max_pages=20, new_pages=20, new=FAKE + 4096, budget=200)
    assert _evict(lib, nwb=400, nwh=200, **kw, **far) == INVALID
    assert _evict(lib, wb=400, wh=200, wk=200, nwb=sb, nwh=sh, **far) == INVALID


def test_weights_in_place_keep_their_strides(lib):
    for nwb, nwh in ((192, 64), (256, 128), (64, 128)):
        assert _evict(lib, wb=128, wh=64, wk=64, nw=FAKE, nwb=nwb, nwh=nwh, budget=64) == INVALID


def test_tables_in_place_keep_their_width(lib):
    """[B, pages] rows of another width would be other sequences' pages."""
    assert _evict(lib, max_pages=5, new_pages=4, nw=FAKE + 4096) == INVALID
    assert _evict(lib, max_pages=4, new_pages=5, nw=FAKE + 4096) == INVALID


def test_evict_refusals_with_weights_elsewhere(lib):
    """Each of the other refusals, in a call that is in order but for it."""
    for kw, code in test_prompt_cpu.test_evict_refusals.pytestmark[0].args[1]:
        assert _evict(lib, **{"nw": FAKE + 4096, **kw}) == code, kw
