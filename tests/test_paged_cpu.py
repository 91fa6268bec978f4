"""Host-side refusals of the paged-cache entry points: they return from validation before any CUDA call."""
import ctypes
import os
import struct

import pytest
import torch

import exact_attention_30_gb300 as fa
from exact_attention_30_gb300 import build as fa_build

FAKE = 0x10000  # an aligned non-null value: never dereferenced, validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fa.library_path()):
        fa_build.build()
    return fa.load_library()


def _cache(**kw):
    c = dict(k=FAKE, v=FAKE, num_pages=10, kv_heads=4, page_size=16, d=128, k_page_stride=8192, k_head_stride=2048,
             k_row_stride=128, v_page_stride=8192, v_head_stride=2048, v_row_stride=128)
    c.update(kw)
    return struct.pack("@PPiiii6q", *c.values())  # fa_paged_kv


BAD_POOLS = [
    (dict(k=0), fa.FA_ERR_INVALID_ARG), (dict(v=0), fa.FA_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), fa.FA_ERR_INVALID_ARG), (dict(v=FAKE + 2), fa.FA_ERR_INVALID_ARG),
    (dict(num_pages=0), fa.FA_ERR_INVALID_ARG), (dict(kv_heads=0), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=0), fa.FA_ERR_INVALID_ARG), (dict(page_size=12), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=65544), fa.FA_ERR_UNSUPPORTED), (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(k_page_stride=8193), fa.FA_ERR_INVALID_ARG), (dict(v_head_stride=2052), fa.FA_ERR_INVALID_ARG),
    (dict(k_row_stride=64), fa.FA_ERR_INVALID_ARG), (dict(v_row_stride=0), fa.FA_ERR_INVALID_ARG),
    (dict(k_head_stride=-2048), fa.FA_ERR_INVALID_ARG), (dict(k_page_stride=1 << 39), fa.FA_ERR_INVALID_ARG),
]


def _append(lib, cache=None, K=FAKE, V=FAKE, ks=512, vs=512, Q=FAKE, Qo=FAKE + 65536, qs=1024, qos=1024, Hq=8,
            tables=FAKE, max_pages=4, lens=FAKE, cu=FAKE, B=2, total=6, cos=FAKE, sin=FAKE, rot=128, max_pos=64,
            positions=None, flags=0, dt=fa.FA_BF16):
    cache = _cache() if cache is None else cache
    return lib.fa_kv_append(K, V, ks, vs, Q, Qo, qs, qos, Hq, cache, tables, max_pages, lens, cu, B,
                            total, cos, sin, rot, max_pos, positions, flags, dt, None)


def _decode(lib, cache=None, Q=FAKE, qs=None, tables=FAKE, max_pages=4, lens=FAKE, O=FAKE, os_=None, LSE=FAKE,
            ws=FAKE, ws_bytes=1 << 40, B=2, Hq=8, Nq=1, scale=0.1, dt=fa.FA_BF16, prefix=None, prefix_len=0,
            shared=False):
    cache = _cache() if cache is None else cache
    st = lambda s: None if s is None else (ctypes.c_longlong * 3)(*s)
    if shared:
        return lib.fa_decode_shared(Q, st(qs), cache, prefix, prefix_len, tables, max_pages, lens, O,
                                    st(os_), LSE, ws, ws_bytes, B, Hq, Nq, scale, dt, None)
    return lib.fa_decode_paged(Q, st(qs), cache, tables, max_pages, lens, O, st(os_), LSE, ws, ws_bytes,
                               B, Hq, Nq, scale, dt, None)


@pytest.mark.parametrize("kw,code", BAD_POOLS)
def test_bad_pools_are_refused_by_every_entry_point(lib, kw, code):
    assert _append(lib, _cache(**kw)) == code
    assert _decode(lib, _cache(**kw)) == code
    assert _decode(lib, _cache(**kw), shared=True, prefix=FAKE, prefix_len=20) == code


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), fa.FA_ERR_INVALID_ARG), (dict(V=0), fa.FA_ERR_INVALID_ARG), (dict(K=FAKE + 4), fa.FA_ERR_INVALID_ARG),
    (dict(Q=0), fa.FA_ERR_INVALID_ARG), (dict(Qo=0), fa.FA_ERR_INVALID_ARG), (dict(Hq=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=-1), fa.FA_ERR_INVALID_ARG), (dict(ks=504), fa.FA_ERR_INVALID_ARG), (dict(vs=513), fa.FA_ERR_INVALID_ARG),
    (dict(qs=1016), fa.FA_ERR_INVALID_ARG), (dict(qos=1028), fa.FA_ERR_INVALID_ARG),
    (dict(Qo=FAKE, qos=2048), fa.FA_ERR_INVALID_ARG), (dict(tables=0), fa.FA_ERR_INVALID_ARG),
    (dict(tables=FAKE + 2), fa.FA_ERR_INVALID_ARG), (dict(max_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(lens=0), fa.FA_ERR_INVALID_ARG), (dict(cu=None, total=7), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_ERR_INVALID_ARG), (dict(total=0), fa.FA_ERR_INVALID_ARG),
    (dict(cos=None), fa.FA_ERR_INVALID_ARG), (dict(sin=FAKE + 4), fa.FA_ERR_INVALID_ARG),
    (dict(max_pos=0), fa.FA_ERR_INVALID_ARG), (dict(rot=-16), fa.FA_ERR_INVALID_ARG),
    (dict(rot=144), fa.FA_ERR_INVALID_ARG), (dict(rot=24), fa.FA_ERR_UNSUPPORTED),
    (dict(positions=FAKE + 2), fa.FA_ERR_INVALID_ARG), (dict(flags=1), fa.FA_ERR_INVALID_ARG),
    (dict(dt=fa.FA_F32), fa.FA_ERR_UNSUPPORTED), (dict(dt=9), fa.FA_ERR_INVALID_ARG),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Q=0), fa.FA_ERR_INVALID_ARG), (dict(O=0), fa.FA_ERR_INVALID_ARG), (dict(LSE=0), fa.FA_ERR_INVALID_ARG),
    (dict(Q=FAKE + 8), fa.FA_ERR_INVALID_ARG), (dict(ws=0), fa.FA_ERR_INVALID_ARG),
    (dict(ws=FAKE + 16), fa.FA_ERR_INVALID_ARG),
    (dict(tables=0), fa.FA_ERR_INVALID_ARG), (dict(lens=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=0), fa.FA_ERR_INVALID_ARG), (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=6), fa.FA_ERR_INVALID_ARG), (dict(Nq=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=64, Nq=5), fa.FA_ERR_UNSUPPORTED), (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), fa.FA_ERR_INVALID_ARG), (dict(dt=fa.FA_F32), fa.FA_ERR_UNSUPPORTED),
    (dict(qs=(1024, 100, 128)), fa.FA_ERR_INVALID_ARG), (dict(os_=(1028, 128, 128)), fa.FA_ERR_INVALID_ARG),
    (dict(Nq=2, qs=(2048, 256, 64)), fa.FA_ERR_INVALID_ARG), (dict(B=1 << 23), fa.FA_ERR_UNSUPPORTED),
])
def test_decode_refusals(lib, kw, code):
    assert _decode(lib, **kw) == code
    assert _decode(lib, shared=True, prefix=FAKE, prefix_len=100, **kw) == code


def test_shared_refusals(lib):
    assert _decode(lib, shared=True, prefix=FAKE, prefix_len=-1) == fa.FA_ERR_INVALID_ARG
    assert _decode(lib, shared=True, prefix=0, prefix_len=5) == fa.FA_ERR_INVALID_ARG
    assert _decode(lib, shared=True, prefix=FAKE, prefix_len=(1 << 30) + 1) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_decode_paged_workspace_bytes(2, 8, 3, 1, 128) == 0
    assert fa.fa_decode_paged_workspace_bytes(2, 8, 4, 33, 128) == 0
    assert fa.fa_decode_shared_workspace_bytes(2, 8, 4, 1, -1, 128) == 0


def test_binding_refuses_before_the_library_is_asked():
    bf = torch.bfloat16
    pool = torch.zeros(4, 2, 16, 64, dtype=bf)
    tables, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 2, 1, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_decode_paged(q, pool, pool, tables, lens)
    with pytest.raises(ValueError, match="prefix_pages is missing"):
        fa.fa_decode_shared(q, pool, pool, None, 5, tables, lens)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_kv_append(torch.zeros(1, 2, 64, dtype=bf), torch.zeros(1, 2, 64, dtype=bf), pool, pool, tables, lens)
    with pytest.raises(TypeError):
        fa.fa_decode_paged(q, None, pool, tables, lens)
    with pytest.raises(ValueError, match="even"):
        fa.fa_rope_tables(10, 3)


def test_rope_tables_hold_far_positions():
    """Angles are formed in fp64: position 10^6 of the fastest pair is exact to fp32 rounding of the result."""
    import numpy as np
    cos, sin = fa.fa_rope_tables(1000001, 16, base=500.0)
    assert cos.shape == (1000001, 8) and cos.dtype == torch.float32
    a = 10.0 ** 6 * 500.0 ** (-2 * np.arange(8) / 16)
    # the angle in fp64 is off by 2^-52 of 10^6 rad, its cosine by no more; then one rounding to fp32
    assert np.abs(cos[-1].double().numpy() - np.cos(a)).max() <= 2.0 ** -25 + 1e-9
    assert np.abs(sin[-1].double().numpy() - np.sin(a)).max() <= 2.0 ** -25 + 1e-9
