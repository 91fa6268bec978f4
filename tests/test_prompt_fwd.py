"""fa_prompt_fwd and fa_prompt_paged on the GPU against the plain definition in fp64, row by row."""
import math

import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache
from prompt_utils import Paged, Prompts, check_forward, offsets

pytestmark = pytest.mark.gpu

LENS = (0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300)


def _fwd(c, scale=None, **kw):
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, c.max_q, c.cu_k, c.max_k, scale=scale, **kw)
    assert fa.fa_check_device_status() == fa.FA_OK
    return o, lse


def _check(c, scale=None, **kw):
    o, lse = _fwd(c, scale, **kw)
    check_forward(c, o, lse, 1 / math.sqrt(c.d) if scale is None else scale)
    return o, lse


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 7, 8, 12, 16, 33, 64, 71, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_lengths_and_groups(g, d):
    hkv = 2 if g <= 8 else 1
    _check(Prompts(LENS, g * hkv, hkv, d, seed=g + d, pad=(3, 5), fused=g % 2 == 0))


@pytest.mark.parametrize("n,m", [(1, 1), (1, 500), (37, 37), (64, 1000), (5, 3), (130, 1), (300, 299), (129, 0), (0, 40),
                                 (200, 456), (1, 0)])
@pytest.mark.parametrize("g", [1, 4, 6])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_of_their_own(n, m, g, d):
    """Cached keys before the tokens; fewer keys than tokens leave rows without a key."""
    c = Prompts((n, 17, n), 2 * g, 2, d, m=(m, 40, m), seed=n + m + g, pad=(1, 130))
    _check(c)


@pytest.mark.parametrize("n,m,g,d", [(20, 5000, 4, 128), (3, 9000, 2, 64), (1, 4000, 1, 128), (40, 2600, 16, 128),
                                     (70, 70, 4, 64)])
def test_key_ranges(n, m, g, d):
    """Few blocks with many keys: split into key ranges, and the same without scratch."""
    c = Prompts((n, 0, 2), g, 1, d, m=(m, 3, 700), seed=m)
    need = fa.fa_prompt_fwd_workspace_bytes(3, g, 1, c.total, c.max_q, c.max_k, d)
    assert need > 0  # the third sequence alone has 700 keys
    o, lse = _check(c)
    whole, lse1 = torch.empty_like(o), torch.empty_like(lse)
    lib = fa.load_library()
    rc = lib.fa_prompt_fwd(c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), g * d, d, d, whole.data_ptr(), g * d,
                           lse1.data_ptr(), c.cu_q.data_ptr(), c.cu_k.data_ptr(), 3, g, 1, c.total, c.total_k, c.max_q,
                           c.max_k, None, 0, d, 1 / math.sqrt(d), fa.FA_BF16, torch.cuda.current_stream().cuda_stream)
    assert rc == fa.FA_OK
    check_forward(c, whole, lse1, 1 / math.sqrt(d))


def test_many_sequences_and_one_long():
    lens = [(7 * i) % 90 for i in range(150)] + [2100]
    c = Prompts(lens, 4, 1, 128, seed=1)
    o, lse = _fwd(c)
    check_forward(c, o, lse, 1 / math.sqrt(128), seqs=range(0, 151, 10))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [(20, 60, 64, 1), (33, 70)])
def test_blocks_of_one_and_of_two_query_tiles_in_turn(lens, d):
    """More blocks than SMs: every CTA takes several, whose query tiles visit different numbers of key tiles, or
    none, some of them many in a row."""
    n = [lens[i % len(lens)] for i in range(150)]
    m = [(700, 1900, 300, 1100, 40)[i % 5] + n[i] for i in range(150)]
    c = Prompts(n, 16, 4, d, m=m, seed=d)
    o, lse = _fwd(c)
    check_forward(c, o, lse, 1 / math.sqrt(d), seqs=range(0, 150, 17))


def test_sums_that_grow_late():
    """The largest scores come last, by far: what was summed before is scaled down, tile after tile."""
    for d in (64, 128):
        c = Prompts((100, 260), 8, 2, d, m=(2000, 900), seed=d)
        for b, rows, keys, nb, mb in c.seqs():
            ramp = torch.linspace(0.02, 3.0, mb, device="cuda")[:, None, None]
            c.k[keys] = (c.k[keys].abs() * ramp).to(torch.bfloat16)
            c.q[rows] = c.q[rows].abs()
        _check(c)


def test_large_scores_and_scale():
    for scale in (0.5, 1.7):
        _check(Prompts((150, 260), 6, 2, 128, seed=3, big=16), scale)


def test_rows_outside_sequences_and_strided_outputs():
    c = Prompts((40, 0, 90), 8, 2, 64, seed=5, pad=(7, 9))
    big = torch.full((c.total, 3, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, c.total), 5.0, device="cuda")
    o, _ = _check(c, out=big[:, 1], lse=lse)
    assert o.data_ptr() == big[:, 1].data_ptr()
    assert (big[:, 0] == 5).all() and (big[:, 2] == 5).all()
    assert (o[:7] == 5).all() and (o[-9:] == 5).all()
    assert (lse[:, :7] == 5).all() and (lse[:, -9:] == 5).all()


def test_keys_behind_a_sequence_have_no_influence():
    """The next sequence's keys, not finite, stand in the last tile of the one before."""
    c = Prompts((50, 70), 4, 1, 128, seed=8)
    ref, ref_l = _fwd(c)
    c.k[50:], c.v[50:] = math.nan, math.inf
    c.q[50:] = math.nan
    o, lse = _fwd(c)
    assert torch.equal(o[:50], ref[:50]) and torch.equal(lse[:, :50], ref_l[:, :50])


def test_bad_offsets_are_left_out():
    c = Prompts((40, 50, 60), 4, 2, 64, seed=9)
    for bad in ([0, 90, 40, 150], [0, 40, 151, 150], [0, -1, 90, 150]):
        cu = torch.tensor(bad, dtype=torch.int32).cuda()
        out, lse = torch.full_like(c.q, 3.0), torch.full((4, 150), 3.0, device="cuda")
        fa.fa_prompt_fwd(c.q, c.k, c.v, cu, 60, cu, 60, out=out, lse=lse)
        assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
        for b in range(3):
            if 0 <= bad[b] <= bad[b + 1] <= 150 and bad[b + 1] - bad[b] <= 60:
                assert (out[bad[b]:bad[b + 1]] != 3).any()
    # longer than the bounds
    fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 59)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_check_device_status() == fa.FA_OK


def test_graph_follows_offsets_and_streams():
    c = Prompts((100, 28, 0), 8, 2, 128, seed=10)
    cu = c.cu_q.clone()
    out, lse = torch.zeros_like(c.q), torch.zeros((8, 128), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.fa_prompt_fwd(c.q, c.k, c.v, cu, 128, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_prompt_fwd(c.q, c.k, c.v, cu, 128, out=out, lse=lse)
    for lens in ((100, 28, 0), (1, 1, 126), (0, 128, 0)):
        cu.copy_(offsets(lens))
        graph.replay()
        torch.cuda.synchronize()
        c.n = c.m = list(lens)
        check_forward(c, out, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 1000])
@pytest.mark.parametrize("g", [1, 4, 7])
@pytest.mark.parametrize("d", [64, 128])
def test_paged(page, g, d):
    lens = (0, 1, 40, 129, 300, 511, 90)
    cache = Cache(lens, 2, page, d, seed=page + g, rows_first=g == 4, width_extra=2)
    cache.poison()
    c = Paged((3, 1, 40, 100, 33, 0, 200), cache, 2 * g, seed=g, pad=(0, 4))
    o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 200)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_forward(c, o, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("n,m", [(70, 6000), (1, 3000), (65, 65)])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_key_ranges(n, m, d):
    cache = Cache((m, n + 2), 1, 16, d, seed=m)
    cache.poison()
    c = Paged((n, n), cache, 4, seed=n)
    o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, n)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_forward(c, o, lse, 1 / math.sqrt(d))


@pytest.mark.parametrize("d", [64, 128])
def test_paged_wide_tables(d):
    """Tables far wider than the sequences: the ranges follow what there is, and nothing is read that no range wrote."""
    cache = Cache((900, 0, 129, 2500), 4, 64, d, seed=d, width_extra=2000)
    c = Paged((60, 0, 129, 3), cache, 16, seed=d, pad=(2, 3))
    most = cache.tables.shape[1] * 64
    n = fa.fa_prompt_fwd_workspace_bytes(4, 16, 4, c.total, 129, most, d)
    assert n > 0
    ws = torch.full((n + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 129, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_forward(c, o, lse, 1 / math.sqrt(d))
    assert (ws[n:] == 255).all()


def test_paged_bad_pages_and_lengths():
    cache = Cache((200, 90), 2, 16, 64, seed=4)
    c = Paged((20, 30), cache, 4)
    for p in (-1, cache.pages, 1 << 30):
        cache.tables[0, 3] = p
        o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 30)
        assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
        check_forward(c, o, lse, 1 / 8, seqs=[1])
    for bad in (-1, cache.tables.shape[1] * 16 + 1):
        lens = torch.tensor([bad, 90], dtype=torch.int32).cuda()
        o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, lens, c.cu_q, 30)
        assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
        check_forward(c, o, lse, 1 / 8, seqs=[1])


def test_refusals():
    c = Prompts((8, 8), 4, 2, 64)
    call = lambda **kw: fa.fa_prompt_fwd(**{**dict(q=c.q, k=c.k, v=c.v, cu_seqlens_q=c.cu_q, max_seqlen_q=8), **kw})
    for kw in (dict(q=c.q.float()), dict(k=c.k.cpu()), dict(v=c.v[:8]), dict(q=c.q[..., ::2]), dict(q=c.q[:, :3]),
               dict(cu_seqlens_q=c.cu_q.long()), dict(cu_seqlens_k=c.cu_k[:2], max_seqlen_k=8),
               dict(cu_seqlens_k=c.cu_k), dict(lse=torch.empty((16, 4), device="cuda")), dict(max_seqlen_q=1 << 40)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(max_seqlen_q=0), dict(max_seqlen_q=17), dict(scale=0.0), dict(scale=math.nan)):
        with pytest.raises(fa.FAError):
            call(**kw)
    # no tokens at all
    o, lse = call(q=c.q[:0], k=c.k[:0], v=c.v[:0], cu_seqlens_q=torch.zeros(3, dtype=torch.int32).cuda())
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
