"""Paged-cache calls at the edge of what the header allows: offsets that do not fit the tokens, scores of -inf, wide tables, sizes
past 32 bits, small boxes, the plain entry of the library, padding in front, captured branches."""
import math

import numpy as np
import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache, check_decode

pytestmark = pytest.mark.gpu


def _call(c, q):
    if c.prefix:
        return fa.fa_decode_shared(q, c.k, c.v, c.prefix_pages, c.prefix, c.tables, c.seq_lens)
    return fa.fa_decode_paged(q, c.k, c.v, c.tables, c.seq_lens)


def _ends_behind(n, last_end):
    """n sequences of one new token each, the last one's end moved."""
    cu = list(range(n + 1))
    cu[-1] = last_end
    return cu


@pytest.mark.parametrize("cu,total,lens", [
    ([0, 2, 4, 7], 6, (30, 20, 10)),          # the last end behind the tokens: its keys would move by one
    ([0, 2, 9, 9], 6, (30, 20, 10)),          # a sequence from the tokens to behind them, an empty one there
    ([-1, 2, 4, 6], 6, (30, 20, 10)),         # a begin before the tokens
    ([0, 2, 2, 1], 6, (30, 20, 10)),          # an end before its begin
    (_ends_behind(40, 43), 40, (17,) * 40),   # more sequences than one round of the search
    (_ends_behind(1100, 1101), 1100, (9,) * 1100),
    ([0, 1500, 2401], 2400, (1501, 1000)),    # a warp for every token
])
def test_tokens_of_inconsistent_offsets_are_not_stored(cu, total, lens):
    """A sequence whose offsets do not lie within the tokens is reported, and its cache and its rows of the queries
    stay; the other sequences' tokens are stored where they belong."""
    hq, hkv, d, page = 4, 2, 64, 16
    c = Cache(lens, hkv, page, d, seed=len(lens), width_extra=1)
    x = torch.randn((total, hq + 2 * hkv, d), generator=torch.Generator().manual_seed(total)).to(torch.bfloat16).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    want_k, want_v = c.k.clone(), c.v.clone()
    out = torch.full((total, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    want_q = out.clone()
    tables = c.tables.cpu()
    for b, n in enumerate(lens):
        if not 0 <= cu[b] <= cu[b + 1] <= total:
            continue
        t = torch.arange(cu[b], cu[b + 1])
        pos = n - cu[b + 1] + t
        pages, rows = tables[b, pos // page].long().cuda(), (pos % page).cuda()
        t = t.cuda()
        want_k[pages, :, rows], want_v[pages, :, rows], want_q[t] = k[t], v[t], q[t]
    fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, torch.tensor(cu, dtype=torch.int32).cuda(), q=q, q_out=out)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_check_device_status() == fa.FA_OK  # cleared
    assert torch.equal(out, want_q)
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)


class _WithoutInfiniteKeys(Cache):
    """What is left of the keys where a row's score of every infinite one is -inf: their weights are zero."""

    def keys_values(self, b, h):
        k, v = super().keys_values(b, h)
        finite = np.isfinite(k).all(1)
        return k[finite], v[finite]

    def spoil(self, table, first, last):
        for j in range(first, last):
            self.k[int(table[j // self.page]), :, j % self.page, 1] = math.inf


@pytest.mark.parametrize("lens,g,prefix,spoiled,own_spoiled", [
    # a prefix's kernel of its own, 80 rows a head: the only key of the last tile (and key range), the first
    # tile, one between, several ranges, all of the prefix
    ((60,) * 20, 4, 129, (128, 129), (0, 0)),
    ((60,) * 20, 4, 300, (0, 128), (0, 0)),
    ((60,) * 20, 4, 300, (128, 256), (0, 0)),
    ((60,) * 20, 4, 1500, (100, 1100), (0, 0)),
    ((60,) * 20, 4, 200, (0, 200), (0, 0)),
    ((300,) * 40, 8, 1000, (0, 900), (0, 200)),  # 320 rows, and own keys
    # the prefix as one more sequence, and none; rows of 8, 16, 32 and two units
    ((200, 70), 4, 500, (0, 300), (0, 64)),
    ((9000, 40), 4, 0, (0, 0), (0, 39)),
    ((9000, 70), 12, 0, (0, 0), (3, 69)),
    ((3000, 400), 24, 0, (0, 0), (0, 390)),
    ((3000, 400), 40, 0, (0, 0), (0, 390)),
])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity_have_no_weight(lens, g, prefix, spoiled, own_spoiled, d):
    """Infinite keys whose scores are -inf in every row count as absent, also where a whole tile, a CTA's share or a
    key range holds nothing else."""
    c = _WithoutInfiniteKeys(lens, 2, 16, d, seed=d + prefix, prefix=prefix)
    q = torch.randn((len(lens), 2 * g, 1, d), generator=torch.Generator().manual_seed(g)).to(torch.bfloat16).cuda()
    q[..., 1] = -q[..., 1].abs() - 0.5
    c.spoil(c.prefix_pages, *spoiled)
    for b in range(len(lens)):
        c.spoil(c.tables[b], *own_spoiled)
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(d), seqs=sorted({0, 1, len(lens) - 1}))


@pytest.mark.parametrize("lens,g,nq,prefix", [((5, 0, 300), 4, 1, 0), ((5, 0, 300), 4, 2, 90), ((90, 0, 700) * 10, 4, 1, 2500),
                                              ((40,) * 33, 8, 1, 700)])
@pytest.mark.parametrize("d", [64, 128])
def test_tables_far_wider_than_the_sequences(lens, g, nq, prefix, d):
    """Tables as wide as a server's longest context, eager and captured, one sequence grown past the others since."""
    c = Cache(lens, 2, 16, d, seed=d + len(lens), prefix=prefix, width_extra=8192)
    c.poison()
    q = torch.randn((len(lens), 2 * g, nq, d), generator=torch.Generator().manual_seed(g)).to(torch.bfloat16).cuda()
    seqs = sorted({0, 1, 2, len(lens) - 1})
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(d), seqs=seqs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = _call(c, q)
    # sequence 1 now names the pages of sequence 2, twice over
    n = -(-c.lens[2] // c.page)
    c.tables[1, :n] = c.tables[2, :n]
    c.tables[1, n:2 * n] = c.tables[2, :n]
    c.lens[1] = c.lens[2] // c.page * c.page
    c.seq_lens[1] = c.lens[1]
    graph.replay()
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(d), seqs=seqs)


def test_sizes_past_32_bits_are_refused():
    """A prefix length and a table's width that 32 bits would cut to small ones of the same call (2^32 + 20, 2^32 + 1)."""
    c = Cache((20, 5), 2, 16, 64, seed=34, prefix=20)
    q = torch.randn((2, 4, 1, 64), device="cuda").to(torch.bfloat16)
    pages = torch.zeros((1 << 16) + 1, dtype=torch.int32, device="cuda")
    pool = torch.zeros((1, 2, 1 << 16, 64), dtype=torch.bfloat16, device="cuda")
    for n in ((1 << 32) + 20, 1 << 31):
        with pytest.raises(ValueError, match="32 bits"):
            fa.fa_decode_shared(q, pool, pool.clone(), pages, n, c.tables, c.seq_lens)
    with pytest.raises(fa.FAError):  # within 32 bits, past what the library takes
        fa.fa_decode_shared(q, pool, pool.clone(), pages, (1 << 30) + 1, c.tables, c.seq_lens)
    wide = torch.empty((1, (1 << 32) + 1), dtype=torch.int32, device="cuda")
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        fa.fa_decode_paged(q[:1], c.k, c.v, wide, c.seq_lens[:1])
    with pytest.raises(ValueError, match="32 bits"):
        fa.fa_kv_append(k, k, c.k, c.v, wide, c.seq_lens[:1])





@pytest.mark.parametrize("page", [8, 24, 40, 200])
@pytest.mark.parametrize("B,g,nq,prefix", [(20, 4, 1, 700), (40, 8, 2, 333), (9, 5, 3, 1000)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_of_many_rows_in_pages_of_odd_multiples_of_8(B, g, nq, prefix, page, d):
    """Boxes of 8 rows in the prefix's kernel."""
    lens = np.random.default_rng(page + B).integers(0, 90, B).tolist()
    c = Cache(lens, 2, page, d, seed=B + page, prefix=prefix, rows_first=page == 24)
    c.poison()
    q = torch.randn((B, 2 * g, nq, d), generator=torch.Generator().manual_seed(page)).to(torch.bfloat16).cuda()
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(d), seqs=sorted({0, 1, B // 2, B - 1}))



@pytest.mark.parametrize("lens,g,nq", [((70, 0, 300), 4, 1), ((900, 33), 5, 3), ((200, 65), 16, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_the_entry_without_a_prefix(lens, g, nq, d):
    """fa_decode_paged of the library itself, dense and strided, gives the bits of fa_decode_shared without a prefix."""
    lib = fa.load_library()
    hkv, B, hq = 2, len(lens), 2 * g
    c = Cache(lens, hkv, 16, d, seed=nq + d)
    q = torch.randn((B, hq, nq, d), generator=torch.Generator().manual_seed(g)).to(torch.bfloat16).cuda()
    want, want_lse = fa.fa_decode_shared(q, c.k, c.v, None, 0, c.tables, c.seq_lens, scale=0.1)
    pool = fa._pack_pool(c.k.data_ptr(), c.v.data_ptr(), c.pages, hkv, c.page, d, *c.k.stride()[:3], *c.v.stride()[:3])
    n = fa.fa_decode_paged_workspace_bytes(B, hq, hkv, nq, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    q_rows = torch.zeros((B, nq, hq + 3, d), dtype=torch.bfloat16, device="cuda")
    q_rows[:, :, :hq] = q.transpose(1, 2)
    o_rows = torch.full_like(q_rows, 7.0)
    strides = lambda t: fa._pack_strides(t.stride(0), t.stride(2), t.stride(1))
    o = torch.empty_like(q)
    for query, q_strides, out, o_strides in ((q, None, o, None), (q_rows, strides(q_rows), o_rows, strides(o_rows))):
        lse = torch.empty((B, hq, nq), dtype=torch.float32, device="cuda")
        assert lib.fa_decode_paged(query.data_ptr(), q_strides, pool, c.tables.data_ptr(), c.tables.shape[1],
                                   c.seq_lens.data_ptr(), out.data_ptr(), o_strides, lse.data_ptr(), ws.data_ptr(), n,
                                   B, hq, nq, 0.1, fa.FA_BF16, torch.cuda.current_stream().cuda_stream) == fa.FA_OK
        assert fa.fa_check_device_status() == fa.FA_OK
        assert torch.equal(lse, want_lse)
    assert torch.equal(o, want)
    assert torch.equal(o_rows[:, :, :hq].transpose(1, 2), want) and bool((o_rows[:, :, hq:] == 7.0).all())



def test_tokens_before_the_first_offset_are_padding():
    """Offsets that begin past the first packed token: what stands before them is left alone, like what stands behind."""
    lens, hq, hkv, d = (20, 9), 4, 2, 64
    c = Cache(lens, hkv, 16, d, seed=3)
    x = torch.randn((9, hq + 2 * hkv, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    want_k, want_v = c.k.clone(), c.v.clone()
    out = torch.full((9, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    for t, b, pos in ((2, 0, 17), (3, 0, 18), (4, 0, 19), (5, 1, 7), (6, 1, 8)):
        page = int(c.tables[b, pos // 16])
        want_k[page, :, pos % 16], want_v[page, :, pos % 16] = k[t], v[t]
    fa.fa_kv_append(k, v, c.k, c.v, c.tables, c.seq_lens, torch.tensor([2, 5, 7], dtype=torch.int32).cuda(), q=q, q_out=out)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.equal(out[2:7], q[2:7]) and bool((out[:2] == 3.0).all()) and bool((out[7:] == 3.0).all())
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)


@pytest.mark.parametrize("prefix", [0, 900])
def test_captured_branches_and_copies(prefix):
    """Calls captured behind a copy of their lengths, in two branches at once, and behind both branches."""
    lens = (100, 33, 70) * 10
    c = Cache(lens, 2, 16, 64, seed=50 + prefix, prefix=prefix)
    q = torch.randn((30, 8, 1, 64), generator=torch.Generator().manual_seed(51)).to(torch.bfloat16).cuda()
    want, want_lse = _call(c, q)
    check_decode(c, q, want, want_lse, 1 / 8, seqs=(0, 1, 29))
    right, side = c.seq_lens.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        c.seq_lens.copy_(right)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got += [_call(c, q), _call(c, q)]
        got += [_call(c, q), _call(c, q)]
        torch.cuda.current_stream().wait_stream(side)
        got.append(_call(c, q))
    for _ in range(3):
        c.seq_lens.fill_(1)
        for o, lse in got:
            o.fill_(9.0)
        graph.replay()
        assert fa.fa_check_device_status() == fa.FA_OK
        for o, lse in got:
            assert torch.equal(o, want) and torch.equal(lse, want_lse)
