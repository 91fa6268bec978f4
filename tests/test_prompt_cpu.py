"""Host-side refusals of the prompt, key-weight and eviction entry points, before any CUDA call."""
import ctypes
import os
import struct

import pytest
import torch

import exact_attention_30_gb300 as fa
from exact_attention_30_gb300 import build as fa_build

FAKE = 0x10000  # an aligned non-null value: never dereferenced, validation fails first
INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fa.library_path()):
        fa_build.build()
    return fa.load_library()


def _cache(**kw):
    c = dict(k=FAKE, v=FAKE, num_pages=10, kv_heads=2, page_size=16, d=128, k_page_stride=4096, k_head_stride=2048,
             k_row_stride=128, v_page_stride=4096, v_head_stride=2048, v_row_stride=128)
    c.update(kw)
    return struct.pack("@PPiiii6q", *c.values())  # fa_paged_kv


def _fwd(lib, Q=FAKE, K=FAKE, V=FAKE, qs=1024, ks=256, vs=256, O=FAKE, os_=1024, LSE=FAKE, cu=FAKE, cuk=FAKE, B=2, Hq=8,
         Hkv=2, t=50, tk=60, mq=30, mk=40, ws=None, d=128, scale=0.1, dt=fa.FA_BF16):
    return lib.fa_prompt_fwd(Q, K, V, qs, ks, vs, O, os_, LSE, cu, cuk, B, Hq, Hkv, t, tk, mq, mk, ws, 0, d, scale, dt, None)


def _paged(lib, cache=None, Q=FAKE, qs=1024, tables=FAKE, max_pages=4, lens=FAKE, O=FAKE, os_=1024, LSE=FAKE, cu=FAKE, B=2,
           Hq=8, t=50, mq=30, ws=None, scale=0.1, dt=fa.FA_BF16):
    return lib.fa_prompt_paged(Q, qs, _cache() if cache is None else cache, tables, max_pages, lens, O, os_, LSE, cu, B, Hq,
                               t, mq, ws, 0, scale, dt, None)


def _bwd(lib, Q=FAKE, K=FAKE, V=FAKE, O=FAKE, dO=FAKE, qs=1024, ks=256, vs=256, os_=1024, dos=1024, LSE=FAKE, dQ=FAKE,
         dK=FAKE, dV=FAKE, dqs=1024, dks=256, dvs=256, cu=FAKE, cuk=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, Hq=8, Hkv=2, t=50,
         tk=60, mq=30, mk=40, d=128, scale=0.1, dt=fa.FA_BF16):
    return lib.fa_prompt_bwd(Q, K, V, O, dO, qs, ks, vs, os_, dos, LSE, dQ, dK, dV, dqs, dks, dvs, cu, cuk, ws, ws_bytes, B,
                             Hq, Hkv, t, tk, mq, mk, d, scale, dt, None)


def _weights(lib, Q=FAKE, K=FAKE, qs=1024, ks=256, LSE=FAKE, W=FAKE, wb=400, wh=200, wk=200, cu=FAKE, cuk=FAKE, B=2, Hq=8,
             Hkv=2, t=50, tk=60, mq=30, mk=40, window=0, d=128, scale=0.1, flags=0, dt=fa.FA_BF16):
    return lib.fa_prompt_key_weights(Q, K, qs, ks, LSE, W, wb, wh, wk, cu, cuk, B, Hq, Hkv, t, tk, mq, mk, window, d, scale,
                                     flags, dt, None)


def _weights_paged(lib, cache=None, Q=FAKE, qs=1024, tables=FAKE, max_pages=4, lens=FAKE, LSE=FAKE, W=FAKE, wb=400, wh=200,
                   wk=200, cu=FAKE, B=2, Hq=8, t=50, mq=30, window=0, scale=0.1, flags=0, dt=fa.FA_BF16):
    return lib.fa_prompt_key_weights_paged(Q, qs, _cache() if cache is None else cache, tables, max_pages, lens, LSE, W, wb,
                                           wh, wk, cu, B, Hq, t, mq, window, scale, flags, dt, None)


def _step(lib, cache=None, Q=FAKE, qs=None, tables=FAKE, max_pages=4, lens=FAKE, LSE=FAKE, W=FAKE, wb=400, wh=200, wk=200,
          B=2, Hq=8, Nq=1, scale=0.1, flags=0, dt=fa.FA_BF16):
    st = None if qs is None else (ctypes.c_longlong * 3)(*qs)
    return lib.fa_decode_key_weights(Q, st, _cache() if cache is None else cache, tables, max_pages, lens, LSE, W, wb, wh, wk,
                                     B, Hq, Nq, scale, flags, dt, None)


def _evict(lib, cache=None, tables=FAKE, max_pages=4, lens=FAKE, new=FAKE, new_pages=4, new_lens=FAKE, W=FAKE, wb=128, wh=64,
           wk=64, nw=FAKE, nwb=80, nwh=40, kept=FAKE, B=2, budget=40, recent=8, dt=fa.FA_BF16):
    return lib.fa_kv_evict(_cache() if cache is None else cache, tables, max_pages, lens, new, new_pages, new_lens, W, wb, wh,
                           wk, nw, nwb, nwh, kept, B, budget, recent, dt, None)


SIZES = [(dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(t=0), INVALID),
         (dict(tk=0), INVALID), (dict(mq=0), INVALID), (dict(mk=0), INVALID), (dict(mq=51), INVALID), (dict(mk=61), INVALID),
         (dict(mq=-1), INVALID), (dict(t=(1 << 30) + 1), UNSUPPORTED), (dict(tk=(1 << 30) + 1), UNSUPPORTED),
         (dict(Hq=129, Hkv=1), UNSUPPORTED), (dict(B=1 << 24), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID),
         (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
         (dict(dt=fa.FA_F32), UNSUPPORTED), (dict(dt=9), INVALID)]


@pytest.mark.parametrize("kw,code", SIZES)
def test_sizes_are_refused_alike(lib, kw, code):
    assert _fwd(lib, **kw) == code
    assert _bwd(lib, **kw) == code
    assert _weights(lib, **kw) == code
    if "scale" not in kw:
        s = dict(B=2, Hq=8, Hkv=2, t=50, tk=60, mq=30, mk=40, d=128, dt=fa.FA_BF16)
        s.update(kw)
        assert lib.fa_prompt_fwd_workspace_bytes(*s.values()) == 0
        assert lib.fa_prompt_bwd_workspace_bytes(*s.values()) == 0


@pytest.mark.parametrize("kw", [dict(Q=0), dict(K=0), dict(cu=0), dict(cuk=0), dict(LSE=0), dict(Q=FAKE + 8),
                                dict(K=FAKE + 2), dict(LSE=FAKE + 2), dict(cu=FAKE + 1), dict(cuk=FAKE + 2), dict(qs=1016),
                                dict(qs=1028), dict(ks=255), dict(ks=-256), dict(qs=1 << 39)])
def test_inputs_are_refused_alike(lib, kw):
    assert _fwd(lib, **kw) == INVALID
    assert _bwd(lib, **kw) == INVALID
    assert _weights(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(V=0), dict(V=FAKE + 4), dict(vs=252), dict(O=0), dict(O=FAKE + 8), dict(os_=1020)])
def test_forward_and_backward_refusals(lib, kw):
    assert _fwd(lib, **kw) == INVALID
    assert _bwd(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dO=0), dict(dQ=0), dict(dK=0), dict(dV=0), dict(dO=FAKE + 8), dict(dQ=FAKE + 4),
                                dict(dK=FAKE + 2), dict(dV=FAKE + 8), dict(dos=1000), dict(dqs=1028), dict(dks=128),
                                dict(dvs=257), dict(ws=0), dict(ws=FAKE + 128)])
def test_backward_refusals(lib, kw):
    assert _bwd(lib, **kw) == INVALID


def test_workspace_refusals(lib):
    assert _fwd(lib, ws=FAKE + 16) == INVALID
    assert _paged(lib, ws=FAKE + 16) == INVALID
    # the statistics and the fp32 sums of dQ are there whatever the GPU
    need = fa.fa_prompt_bwd_workspace_bytes(2, 8, 2, 50, 60, 30, 40, 128)
    assert need >= 2 * 128 * (128 + 2) * 4
    assert _bwd(lib, ws_bytes=need - 1) == INVALID


@pytest.mark.parametrize("kw,code", [(dict(W=0), INVALID), (dict(W=FAKE + 2), INVALID), (dict(window=-1), INVALID),
                                     (dict(flags=1), INVALID), (dict(flags=8), INVALID), (dict(wk=0), INVALID),
                                     (dict(wh=199), INVALID), (dict(wb=199), INVALID)])
def test_weight_refusals(lib, kw, code):
    assert _weights(lib, **kw) == code
    assert _weights_paged(lib, **kw) == code
    if "window" not in kw:
        assert _step(lib, **kw) == code


PAGED = [(dict(tables=0), INVALID), (dict(tables=FAKE + 2), INVALID), (dict(lens=0), INVALID), (dict(lens=FAKE + 1), INVALID),
         (dict(max_pages=0), INVALID), (dict(max_pages=-3), INVALID), (dict(B=0), INVALID), (dict(dt=fa.FA_F32), UNSUPPORTED)]
POOLS = [(dict(k=0), INVALID), (dict(v=FAKE + 2), INVALID), (dict(num_pages=0), INVALID), (dict(kv_heads=0), INVALID),
         (dict(page_size=12), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(k_row_stride=64), INVALID),
         (dict(v_page_stride=4097), INVALID), (dict(k_head_stride=-2048), INVALID)]


@pytest.mark.parametrize("call", [_paged, _weights_paged, _step, _evict])
def test_paged_refusals(lib, call):
    for kw, code in PAGED:
        assert call(lib, **kw) == code, kw
    for kw, code in POOLS:
        assert call(lib, _cache(**kw)) == code, kw


@pytest.mark.parametrize("kw,code", [(dict(Q=0), INVALID), (dict(Q=FAKE + 8), INVALID), (dict(LSE=0), INVALID),
                                     (dict(Hq=3), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID)])
def test_paged_query_refusals(lib, kw, code):
    assert _paged(lib, **kw) == code
    assert _weights_paged(lib, **kw) == code
    assert _step(lib, **kw) == code


def test_paged_prompt_and_step_refusals(lib):
    for call in (_paged, _weights_paged):
        assert call(lib, qs=1020) == INVALID
        assert call(lib, cu=0) == INVALID
        assert call(lib, mq=51) == INVALID
        assert call(lib, t=0, mq=0) == INVALID
        assert call(lib, Hq=2 * 129) == UNSUPPORTED
    assert _paged(lib, O=0) == INVALID
    assert _paged(lib, os_=1032 - 4) == INVALID
    assert _step(lib, Nq=0) == INVALID
    assert _step(lib, Hq=8, Nq=17) == UNSUPPORTED  # 68 rows to a K/V head
    assert _step(lib, qs=(1024, 100, 128)) == INVALID


@pytest.mark.parametrize("kw,code", [(dict(new=0), INVALID), (dict(new=FAKE + 2), INVALID), (dict(new_lens=0), INVALID),
                                     (dict(W=0), INVALID), (dict(nw=0), INVALID), (dict(kept=0), INVALID),
                                     (dict(kept=FAKE + 2), INVALID), (dict(budget=0), INVALID), (dict(recent=-1), INVALID),
                                     (dict(recent=41), INVALID), (dict(wh=63), INVALID), (dict(wb=63), INVALID),
                                     (dict(nwh=39), INVALID), (dict(nwb=39), INVALID), (dict(new_pages=0), INVALID),
                                     (dict(new_pages=2), INVALID), (dict(budget=(1 << 30) + 1, nwh=64, nwb=128), UNSUPPORTED),
                                     (dict(B=65536), UNSUPPORTED)])
def test_evict_refusals(lib, kw, code):
    assert _evict(lib, **kw) == code


def test_binding_refuses_before_the_library_is_asked():
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(5, 4, 64, dtype=bf), torch.zeros(5, 2, 64, dtype=bf)
    pool = torch.zeros(4, 2, 16, 64, dtype=bf)
    cu, tables, lens = torch.tensor([0, 5], dtype=i32), torch.zeros(1, 2, dtype=i32), torch.ones(1, dtype=i32)
    lse, w = torch.zeros(4, 5), torch.zeros(1, 2, 40)
    for call in (lambda: fa.fa_prompt_fwd(q, k, k, cu, 5), lambda: fa.fa_prompt_paged(q, pool, pool, tables, lens, cu, 5),
                 lambda: fa.fa_prompt_bwd(q, k, k, q, q, lse, cu, 5),
                 lambda: fa.fa_prompt_key_weights(q, k, lse, w, cu, 5),
                 lambda: fa.fa_prompt_key_weights_paged(q, pool, tables, lens, lse, w, cu, 5),
                 lambda: fa.fa_decode_key_weights(q[None, :, :1], pool, tables, lens, lse[None], w),
                 lambda: fa.fa_kv_evict(pool, pool, tables, lens, w, 10)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
