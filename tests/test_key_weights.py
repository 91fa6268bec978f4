"""fa_prompt_key_weights, its paged form and fa_decode_key_weights against the plain definition in fp64, key by key."""
import math

import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache
from prompt_utils import Paged, Prompts, bf16_randn, check_weights, offsets

pytestmark = pytest.mark.gpu

LENS = (0, 1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 300, 600)


def _weights(c, keys, seed):
    return torch.rand((len(c.n), c.hkv, keys), generator=torch.Generator().manual_seed(seed)).cuda()


def _check(c, window=0, accumulate=True, scale=None, extra=3):
    _, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, c.max_q, c.cu_k, c.max_k, scale=scale)
    w = _weights(c, c.max_k + extra, 5)
    before = w.clone()
    got = fa.fa_prompt_key_weights(c.q, c.k, lse, w, c.cu_q, c.max_q, c.cu_k, c.max_k, window=window,
                                   accumulate=accumulate, scale=scale)
    assert got is w and fa.fa_check_device_status() == fa.FA_OK
    check_weights(c, w, before, lse, 1 / math.sqrt(c.d) if scale is None else scale, window, accumulate)
    return w


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 7, 8, 12, 16, 33, 64, 71, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_lengths_and_groups(g, d):
    hkv = 2 if g <= 8 else 1
    _check(Prompts(LENS, g * hkv, hkv, d, seed=g + d, pad=(3, 5), fused=g % 2 == 0))


@pytest.mark.parametrize("window", [1, 7, 32, 33, 64, 100, 128, 1000])
@pytest.mark.parametrize("g,d", [(1, 128), (4, 128), (6, 64)])
def test_windows(window, g, d):
    _check(Prompts((0, 1, 40, 129, 520, 700), 2 * g, 2, d, m=(3, 1, 90, 300, 520, 900), seed=window), window)


@pytest.mark.parametrize("n,m", [(1, 1), (1, 500), (64, 1000), (5, 3), (130, 1), (300, 299), (129, 0), (0, 40), (200, 456)])
@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("g,d", [(4, 128), (3, 64)])
def test_keys_of_their_own(n, m, accumulate, g, d):
    _check(Prompts((n, 17, n), 2 * g, 2, d, m=(m, 40, m), seed=n + m + g, pad=(1, 130)), accumulate=accumulate)


def test_many_units_and_large_scores():
    _check(Prompts((3000, 1700), 8, 4, 128, seed=3, big=16))
    _check(Prompts([(11 * i) % 300 for i in range(150)], 2, 1, 64, seed=4))


def test_other_sequences_have_no_influence():
    c = Prompts((50, 70), 4, 1, 128, seed=8)
    _, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 70)
    ref = fa.fa_prompt_key_weights(c.q, c.k, lse, torch.zeros((2, 1, 70), device="cuda"), c.cu_q, 70)
    c.q[50:], c.k[50:], lse[:, 50:] = math.nan, math.inf, math.nan
    got = fa.fa_prompt_key_weights(c.q, c.k, lse, torch.zeros((2, 1, 70), device="cuda"), c.cu_q, 70)
    assert torch.equal(got[0], ref[0])


@pytest.mark.parametrize("page", [8, 24, 64, 1000])
@pytest.mark.parametrize("g,d,window", [(1, 128, 0), (4, 128, 50), (7, 64, 0)])
def test_prompt_paged(page, g, d, window):
    cache = Cache((0, 1, 40, 129, 300, 511, 90, 1300), 2, page, d, seed=page + g, rows_first=g == 4, width_extra=2)
    cache.poison()
    c = Paged((3, 1, 40, 100, 33, 0, 200, 7), cache, 2 * g, seed=g, pad=(0, 4))
    _, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 200)
    w = _weights(c, 1400, 6)
    before = w.clone()
    fa.fa_prompt_key_weights_paged(c.q, cache.k, cache.tables, cache.seq_lens, lse, w, c.cu_q, 200, window=window)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_weights(c, w, before, lse, 1 / math.sqrt(d), window)


def _step(cache, hq, nq, seed, accumulate=True, w=None, strided=False):
    """A decoding step's weights, checked as prompts of nq tokens each."""
    B = len(cache.lens)
    q = bf16_randn((B, nq, hq, cache.d), seed)
    c = Paged([nq] * B, cache, hq)
    c.q = q.reshape(B * nq, hq, cache.d)
    q4 = q.transpose(1, 2) if strided else q.transpose(1, 2).contiguous()
    _, lse = fa.fa_decode_paged(q4, cache.k, cache.v, cache.tables, cache.seq_lens)
    w = _weights(c, max(cache.lens) + 5, 7) if w is None else w
    before = w.clone()
    got = fa.fa_decode_key_weights(q4, cache.k, cache.tables, cache.seq_lens, lse, w, accumulate=accumulate)
    assert got is w and fa.fa_check_device_status() == fa.FA_OK
    check_weights(c, w, before, lse.transpose(0, 1).reshape(hq, B * nq), 1 / math.sqrt(cache.d), accumulate=accumulate)


@pytest.mark.parametrize("g,nq", [(1, 1), (4, 1), (5, 1), (8, 1), (16, 1), (1, 2), (4, 3), (3, 3), (7, 2), (16, 2), (8, 4),
                                  (64, 1), (8, 8), (1, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_groups_and_new_tokens(g, nq, d):
    cache = Cache((0, 1, 3, 31, 32, 33, 64, 66, 130, 257, 1000), 2, 16, d, seed=g * nq + d, rows_first=g % 2 == 0)
    cache.poison()
    _step(cache, 2 * g, nq, g + nq, accumulate=nq % 2 == 1, strided=g % 2 == 1)


@pytest.mark.parametrize("page", [8, 24, 48, 128, 1000])
def test_decode_pages_and_many_sequences(page):
    cache = Cache([(37 * i) % 400 for i in range(90)] + [5000, 0, 0, 17], 3, page, 128, seed=page)
    cache.poison()
    _step(cache, 6, 1, page)


def test_bad_lengths_pages_and_narrow_rows():
    cache = Cache((200, 90), 2, 16, 64, seed=4)
    q = bf16_randn((2, 4, 1, 64), 1)
    _, lse = fa.fa_decode_paged(q, cache.k, cache.v, cache.tables, cache.seq_lens)
    ref = fa.fa_decode_key_weights(q, cache.k, cache.tables, cache.seq_lens, lse, torch.zeros((2, 2, 200), device="cuda"))
    run = lambda lens, width: fa.fa_decode_key_weights(q, cache.k, cache.tables, lens, lse,
                                                       torch.zeros((2, 2, width), device="cuda"))
    for bad in (-1, cache.tables.shape[1] * 16 + 1):
        got = run(torch.tensor([bad, 90], dtype=torch.int32).cuda(), 300)
        assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
        assert (got[0] == 0).all() and torch.equal(got[1, :, :90], ref[1, :, :90])
    got = run(cache.seq_lens, 199)  # the first sequence does not fit
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert (got[0] == 0).all() and torch.equal(got[1, :, :90], ref[1, :, :90])
    cu = offsets((1, 1))
    got = torch.zeros((2, 2, 199), device="cuda")
    fa.fa_prompt_key_weights_paged(q[:, :, 0], cache.k, cache.tables, cache.seq_lens, lse[..., 0].T.contiguous(), got, cu, 1)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert (got[0] == 0).all() and (got[1, :, :90] > 0).all()
    for p in (-1, cache.pages, 1 << 30):
        cache.tables[0, 3] = p
        got = run(cache.seq_lens, 200)
        assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(got[1], ref[1])


def test_refusals():
    c = Prompts((8, 8), 4, 2, 64)
    _, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 8)
    w = torch.zeros((2, 2, 8), device="cuda")
    call = lambda **kw: fa.fa_prompt_key_weights(**{**dict(q=c.q, k=c.k, lse=lse, weights=w, cu_seqlens_q=c.cu_q,
                                                           max_seqlen_q=8), **kw})
    for kw in (dict(weights=w.double()), dict(weights=w[:1]), dict(weights=w.transpose(1, 2).contiguous().transpose(1, 2)),
               dict(lse=lse[:3]), dict(weights=w.cpu()), dict(window=1 << 40)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(window=-1), dict(scale=0.0), dict(weights=w[:1].expand(2, 2, 8)), dict(max_seqlen_q=0)):
        with pytest.raises(fa.FAError):
            call(**kw)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_wide_tables(d):
    """Tables and rows of weights far wider than the sequences."""
    cache = Cache((900, 0, 129, 2500, 5000), 4, 64, d, seed=d, width_extra=4000)
    c = Paged((60, 0, 129, 3, 700), cache, 16, seed=d, pad=(2, 3))
    o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 700)
    for window in (0, 20):
        w = torch.rand((5, 4, cache.tables.shape[1] * 64), device="cuda")
        before = w.clone()
        fa.fa_prompt_key_weights_paged(c.q, cache.k, cache.tables, cache.seq_lens, lse, w, c.cu_q, 700, window=window)
        assert fa.fa_check_device_status() == fa.FA_OK
        check_weights(c, w, before, lse, 1 / math.sqrt(d), window)
