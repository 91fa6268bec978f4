"""Paged-cache calls at the edge of what the header allows: offsets that do not fit the tokens, scores of -inf, wide tables, sizes
past 32 bits."""
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
