"""fa_kv_append on the GPU against the rotation's definition in fp64; every other element of the pool stays as it was."""
import numpy as np
import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache, check_rotated, to64

pytestmark = pytest.mark.gpu


def _tokens(total, hq, hkv, d, seed, fused=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((total, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _check(c, before_k, before_v, new, starts, q, k, v, got_q, cos, sin, inter, positions=None, skip=()):
    """`new` tokens of each sequence from packed token `starts` on; sequences in `skip` must not have moved."""
    k64, v64, q64 = to64(k), to64(v), None if q is None else to64(q)
    want_k, want_v = to64(before_k), to64(before_v)
    got_k, got_v = to64(c.k), to64(c.v)
    gq = None if got_q is None else to64(got_q)
    none = np.zeros((0,))
    for b, n in enumerate(new):
        for i in range(n if b not in skip else 0):
            t, pos = starts[b] + i, c.lens[b] - n + i
            page, row = int(c.tables[b, pos // c.page]), pos % c.page
            p = pos if positions is None else int(positions[t])
            cc, ss = (none, none) if cos is None else (to64(cos[p]), to64(sin[p]))
            check_rotated(got_k[page, :, row], k64[t], cc, ss, inter, (b, i, "k"))
            if gq is not None:
                check_rotated(gq[t], q64[t], cc, ss, inter, (b, i, "q"))
            want_k[page, :, row] = got_k[page, :, row]
            want_v[page, :, row] = v64[t]
    assert np.array_equal(got_k, want_k)  # nothing else moved
    assert np.array_equal(got_v, want_v)


CASES = [
    # lens after, new tokens, page, hq, hkv, d, rot, interleaved, rows first, fused
    ((1,), (1,), 16, 4, 4, 128, 128, False, False, True),
    ((700,), (1,), 16, 32, 8, 128, 128, False, False, True),
    ((17, 16, 33, 5), (1, 1, 1, 1), 16, 8, 2, 64, 64, True, False, True),
    ((40, 9, 100), (40, 3, 77), 8, 6, 3, 64, 32, True, True, False),
    ((130, 64, 65, 63), (70, 64, 1, 5), 64, 5, 1, 128, 16, False, True, True),
    ((50, 20, 30), (0, 20, 0), 48, 7, 7, 128, 64, False, False, True),
    ((31, 7), (31, 7), 32, 2, 1, 64, 0, False, False, True),
    ((900, 1300), (900, 1000), 256, 32, 8, 128, 128, False, False, True),
    ((700, 333), (555, 333), 128, 16, 16, 64, 48, True, True, True),
]


@pytest.mark.parametrize("lens,new,page,hq,hkv,d,rot,inter,rows_first,fused", CASES)
def test_append_against_the_definition(lens, new, page, hq, hkv, d, rot, inter, rows_first, fused):
    c = Cache(lens, hkv, page, d, seed=sum(lens) + d, rows_first=rows_first, width_extra=2)
    cu = np.concatenate([[0], np.cumsum(new)])
    q, k, v = _tokens(int(cu[-1]), hq, hkv, d, seed=d + rot, fused=fused)
    cos, sin = (None, None) if rot == 0 else fa.fa_rope_tables(max(lens), rot, device="cuda")
    bk, bv = c.k.clone(), c.v.clone()
    out = fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, torch.tensor(cu, dtype=torch.int32).cuda(), q=q,
                          cos=cos, sin=sin, interleaved=inter)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert out.is_contiguous() and out.shape == q.shape
    _check(c, bk, bv, new, cu[:-1], q, k, v, out, cos, sin, inter)


@pytest.mark.parametrize("lens,hq,hkv,d,rot,inter", [((1500, 900, 77), 5, 3, 64, 64, False), ((2100,), 6, 1, 128, 96, True)])
def test_a_warp_for_every_token(lens, hq, hkv, d, rot, inter):
    """More than 2048 new tokens: a token's heads in one warp, the last pass of it partly idle."""
    c = Cache(lens, hkv, 64, d, seed=d)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = _tokens(int(cu[-1]), hq, hkv, d, seed=d + 1)
    cos, sin = fa.fa_rope_tables(max(lens), rot, device="cuda")
    bk, bv = c.k.clone(), c.v.clone()
    out = fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, torch.tensor(cu, dtype=torch.int32).cuda(), q=q,
                          cos=cos, sin=sin, interleaved=inter)
    assert fa.fa_check_device_status() == fa.FA_OK
    _check(c, bk, bv, lens, cu[:-1], q, k, v, out, cos, sin, inter)


def test_equal_counts_without_offsets_keys_only_and_positions():
    lens, new, hkv, d = (20, 33, 3), (3, 3, 3), 2, 128
    c = Cache(lens, hkv, 16, d, seed=1, one_tensor=True)
    _, k, v = _tokens(9, 4, hkv, d, seed=2)
    cos, sin = fa.fa_rope_tables(5000, d, device="cuda")
    pos = torch.randint(0, 5000, (9,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    bk, bv = c.k.clone(), c.v.clone()
    assert fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, cos=cos, sin=sin, positions=pos) is None
    assert fa.fa_check_device_status() == fa.FA_OK
    _check(c, bk, bv, new, (0, 3, 6), None, k, v, None, cos, sin, False, positions=pos)


def test_queries_in_place_and_padding_left_alone():
    """Tokens behind the last sequence and those of a sequence of length zero are neither read nor written."""
    lens, new, hq, hkv, d = (12, 0, 40), (2, 1, 3), 8, 2, 64
    c = Cache(lens, hkv, 16, d, seed=5)
    q, k, v = _tokens(10, hq, hkv, d, seed=6)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    k[6:], v[6:], q[6:] = float("nan"), float("nan"), 7.0
    cos, sin = fa.fa_rope_tables(64, d, device="cuda")
    cu = torch.tensor([0, 2, 3, 6], dtype=torch.int32).cuda()
    bk, bv = c.k.clone(), c.v.clone()
    got = fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, cu, q=q, cos=cos, sin=sin, q_out=q)
    assert got is q and fa.fa_check_device_status() == fa.FA_OK
    assert (q[6:] == 7.0).all() and torch.equal(q[2], q0[2])
    _check(c, bk, bv, new, (0, 2, 3), q0, k0, v0, q, cos, sin, False, skip=(1,))


@pytest.mark.parametrize("break_it", ["page", "page_high", "length", "negative", "position", "offsets", "order"])
def test_bad_contents_are_reported_and_touch_nothing(break_it):
    """One sequence's page, length or position is wrong: it is skipped and reported, its neighbours are appended."""
    lens, new, hq, hkv, d = (30, 20, 10), (2, 2, 2), 4, 2, 128
    c = Cache(lens, hkv, 16, d, seed=7)
    q, k, v = _tokens(6, hq, hkv, d, seed=8)
    cos, sin = fa.fa_rope_tables(64, d, device="cuda")
    cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32).cuda()
    tables, seq_lens, positions = c.tables.clone(), c.seq_lens.clone(), None
    skip = (1,)
    if break_it == "page":
        tables[1, 1] = -1
    elif break_it == "page_high":
        tables[1, 1] = c.pages
    elif break_it == "length":
        seq_lens[1] = 16 * tables.shape[1] + 2
    elif break_it == "negative":
        seq_lens[1] = -5
    elif break_it == "position":
        positions = torch.tensor([28, 29, 64, -1, 8, 9], dtype=torch.int32).cuda()
    elif break_it == "offsets":
        cu[3] = 7
        skip = (2,)
    else:
        cu = torch.tensor([0, 2, 2, 1], dtype=torch.int32).cuda()
        skip = (1, 2)
    bk, bv = c.k.clone(), c.v.clone()
    out = torch.full_like(q, 3.0, memory_format=torch.contiguous_format)
    fa.fa_kv_append(k, v, c.k, c.v, tables, seq_lens, cu, q=q, cos=cos, sin=sin, positions=positions, q_out=out)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_check_device_status() == fa.FA_OK  # cleared
    if break_it in ("offsets", "order"):  # which tokens of bad offsets are taken is not defined
        touched = to64(c.k) != to64(bk)
        ok = {int(p) for p in c.tables.flatten().tolist() if p >= 0}
        assert set(np.nonzero(touched)[0].tolist()) <= ok
        return
    for b in skip:
        assert (out[2 * b:2 * b + 2] == 3.0).all()
    _check(c, bk, bv, new, (0, 2, 4), q, k, v, torch.where((out == 3.0), q, out), cos, sin, False, positions=positions,
           skip=skip)


def test_many_sequences_find_their_tokens():
    """More sequences than one round of the search covers, empty ones among them."""
    rng = np.random.default_rng(0)
    new = rng.integers(0, 4, 1500)
    lens = new + rng.integers(1, 30, 1500)
    hkv, d = 1, 64
    c = Cache(lens.tolist(), hkv, 8, d, seed=9)
    cu = np.concatenate([[0], np.cumsum(new)])
    total = int(cu[-1])
    _, k, v = _tokens(total, 0, hkv, d, seed=10)
    fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, torch.tensor(cu, dtype=torch.int32).cuda())
    assert fa.fa_check_device_status() == fa.FA_OK
    t = np.arange(total)
    seq = np.searchsorted(cu[1:], t, side="right")
    pos = lens[seq] - (cu[seq + 1] - t)
    pages = c.tables.cpu().numpy()[seq, pos // 8]
    assert np.array_equal(to64(c.k)[pages, :, pos % 8], to64(k)) and np.array_equal(to64(c.v)[pages, :, pos % 8], to64(v))


def test_pool_offsets_beyond_32_bits():
    """A page whose elements lie past 2^32 of the pool's start."""
    page, hkv, d = 256, 8, 128
    pages = (1 << 32) // (page * hkv * d) + 2
    k_pool = torch.empty((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v_pool = torch.empty_like(k_pool)
    tables = torch.tensor([[pages - 1]], dtype=torch.int32).cuda()
    lens = torch.tensor([page], dtype=torch.int32).cuda()
    _, k, v = _tokens(page, 0, hkv, d, seed=11)
    fa.fa_kv_append(k, v, k_pool, v_pool, tables, lens)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.equal(k_pool[-1].transpose(0, 1), k) and torch.equal(v_pool[-1].transpose(0, 1), v)


def test_captured_append_follows_its_lengths():
    """A captured step replayed after the lengths and offsets moved."""
    lens, hq, hkv, d = [5, 9], 4, 2, 64
    c = Cache((64, 64), hkv, 16, d, seed=12)
    c.lens = lens
    seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    q, k, v = _tokens(2, hq, hkv, d, seed=13)
    q_out = torch.empty((2, hq, d), dtype=torch.bfloat16, device="cuda")
    cos, sin = fa.fa_rope_tables(64, d, device="cuda")
    call = lambda: fa.fa_kv_append(k, v, c.k, c.v, c.tables, seq_lens, cu, q=q, cos=cos, sin=sin, q_out=q_out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        c.lens = [n + step for n in lens]
        seq_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        bk, bv = c.k.clone(), c.v.clone()
        graph.replay()
        assert fa.fa_check_device_status() == fa.FA_OK
        _check(c, bk, bv, (1, 1), (0, 1), q, k, v, q_out, cos, sin, False)


def test_append_refuses_what_it_cannot_do():
    c = Cache((20,), 2, 16, 64, seed=14)
    q, k, v = _tokens(1, 4, 2, 64, seed=15)
    cos, sin = fa.fa_rope_tables(32, 64, device="cuda")
    a = dict(k=k, v=v, k_pages=c.k, v_pages=c.v, block_tables=c.tables, seq_lens=c.seq_lens)
    for kw in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=v[:, :, :32]), dict(k_pages=c.k.float()),
               dict(v_pages=c.v[:1]), dict(k_pages=c.k.transpose(2, 3)), dict(seq_lens=c.seq_lens.long()),
               dict(block_tables=c.tables[0]), dict(seq_lens=torch.cat([c.seq_lens, c.seq_lens])), dict(cos=cos),
               dict(cos=cos, sin=sin[:5]), dict(cos=cos.double(), sin=sin.double()), dict(q_out=q),
               dict(q=q, q_out=q[:, :2]), dict(q=q.expand(3, 4, 64)), dict(positions=torch.zeros(2, dtype=torch.int32).cuda()),
               dict(cu_seqlens=torch.zeros(3, dtype=torch.int32).cuda())):
        with pytest.raises(ValueError):
            fa.fa_kv_append(**{**a, **kw})
    with pytest.raises(fa.FAError):  # pages of 12 rows
        fa.fa_kv_append(**{**a, "k_pages": c.k[:, :, :12], "v_pages": c.v[:, :, :12]})
