"""fa_decode_paged and fa_decode_shared on the GPU against the plain definition in fp64, row by row."""
import math

import numpy as np
import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache, check_decode, to64

pytestmark = pytest.mark.gpu


def _q(B, hq, nq, d, seed):
    return torch.randn((B, hq, nq, d), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _call(c, q, scale=None, **kw):
    if c.prefix:
        return fa.fa_decode_shared(q, c.k, c.v, c.prefix_pages, c.prefix, c.tables, c.seq_lens, scale, **kw)
    return fa.fa_decode_paged(q, c.k, c.v, c.tables, c.seq_lens, scale, **kw)


def _run(c, hq, nq, seed, scale=None, **kw):
    q = _q(len(c.lens), hq, nq, c.d, seed)
    o, lse = _call(c, q, scale, **kw)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(c.d) if scale is None else scale)
    return q, o, lse


LENS = (0, 1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 300)


@pytest.mark.parametrize("page", [8, 16, 24, 48, 64, 128, 256, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_lengths_and_page_sizes(page, d):
    c = Cache(LENS, 2, page, d, seed=page + d, width_extra=1)
    c.poison()
    _run(c, 8, 1, seed=page)


@pytest.mark.parametrize("g,nq", [(1, 1), (4, 1), (5, 1), (16, 1), (1, 2), (4, 3), (7, 2), (16, 2), (8, 4), (11, 3),
                                  (7, 7), (64, 1), (8, 8), (1, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_and_new_tokens(g, nq, d):
    """Every share of rows of a K/V head; sequences shorter than their new tokens leave rows without a key."""
    c = Cache((0, 1, 3, 64, 66, 130, 257), 2, 16, d, seed=g * nq + d, rows_first=g % 2 == 0)
    c.poison()
    _run(c, 2 * g, nq, seed=g + nq)


@pytest.mark.parametrize("prefix", [1, 15, 16, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_lengths(prefix, d):
    c = Cache((0, 1, 40, 64, 100), 2, 16, d, seed=prefix + d, prefix=prefix)
    c.poison()
    _run(c, 8, 1, seed=prefix)


@pytest.mark.parametrize("B,g,nq,prefix,page", [
    (1, 1, 1, 500, 16), (3, 5, 1, 333, 8), (2, 4, 5, 777, 48), (16, 4, 1, 200, 64), (17, 4, 1, 600, 16),
    (32, 4, 1, 1500, 64), (33, 7, 1, 640, 128), (40, 8, 3, 300, 32), (70, 2, 2, 129, 256), (9, 64, 1, 1100, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_share_a_prefix(B, g, nq, prefix, page, d):
    rng = np.random.default_rng(B + g)
    lens = rng.integers(0, 150, B).tolist()
    c = Cache(lens, 2, page, d, seed=B + d, prefix=prefix, rows_first=B % 2 == 1)
    c.poison()
    _run(c, 2 * g, nq, seed=B)


@pytest.mark.parametrize("g,nq", [(1, 1), (2, 1), (3, 1), (4, 1), (8, 1), (5, 3), (8, 2), (8, 4), (33, 1), (5, 8), (8, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_units_cut_between_ctas(g, nq, d):
    """A long sequence whose keys many CTAs share, short ones, empty ones: rows of one to many parts to merge."""
    c = Cache((6000, 0, 5, 129, 900, 0), 3, 64, d, seed=g + nq)
    c.poison()
    q = _q(6, 3 * g, nq, d, seed=nq)
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(d), heads=[0, 2])


@pytest.mark.parametrize("g,nq", [(6, 2), (8, 4), (9, 5)])
def test_many_cut_units(g, nq):
    """More units than CTAs, of lengths that leave nearly every CTA with a cut one."""
    rng = np.random.default_rng(g)
    lens = rng.integers(1, 400, 150).tolist()
    c = Cache(lens, 3, 16, 64, seed=g)
    q = _q(150, 3 * g, nq, 64, seed=g)
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / 8, heads=[1], seqs=range(0, 150, 7))


@pytest.mark.parametrize("B,g,nq,prefix", [(5, 8, 1, 700), (12, 1, 5, 300), (20, 33, 1, 500), (3, 8, 8, 1500)])
@pytest.mark.parametrize("d", [64, 128])
def test_more_than_32_rows_with_a_prefix(B, g, nq, prefix, d):
    """33 to 64 rows of the batch, and of one sequence."""
    lens = np.random.default_rng(B).integers(0, 500, B).tolist()
    c = Cache(lens, 2, 32, d, seed=B + d, prefix=prefix)
    c.poison()
    q = _q(B, 2 * g, nq, d, seed=B)
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / math.sqrt(d), seqs=sorted({0, 1, B // 2, B - 1}))


def test_one_long_sequence_among_short_ones():
    c = Cache((5, 20000, 1, 300, 64), 2, 64, 128, seed=1)
    _run(c, 8, 1, seed=2)


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    c = Cache(rng.integers(0, 40, 700).tolist(), 2, 8, 64, seed=3)
    _run(c, 2, 1, seed=4)


def test_more_sequences_than_threads_and_long_prefix():
    rng = np.random.default_rng(5)
    c = Cache(rng.integers(0, 20, 300).tolist(), 1, 16, 128, seed=5, prefix=3000)
    _run(c, 3, 1, seed=6)


@pytest.mark.parametrize("prefix", [0, 900])
def test_growing_scores_move_the_maximum(prefix):
    """Later keys dominate, then a huge one: the running maximum moves through the whole length."""
    c = Cache((1500, 700), 2, 16, 128, seed=7, prefix=prefix)
    c.k.mul_(torch.linspace(0.05, 6.0, c.pages, device="cuda").view(-1, 1, 1, 1).to(torch.bfloat16))
    c.k[int(c.tables[0, 40]), :, 3] *= 30
    _run(c, 8, 1, seed=8, scale=0.3)


def test_very_negative_scores_are_not_masked():
    """Scores near -1e4 everywhere: nothing of a row underflows to an empty one."""
    c = Cache((100, 33), 1, 16, 64, seed=9, prefix=70)
    c.k.abs_().mul_(8)
    q = -_q(2, 4, 1, 64, 10).abs() * 8
    o, lse = _call(c, q, 4.0)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 4.0)
    assert float(lse.max()) < -1e3


@pytest.mark.parametrize("prefix", [0, 200])
def test_unseen_new_tokens_may_hold_anything(prefix):
    """NaN and infinities in the newest key and value reach the newest query only."""
    c = Cache((150, 65), 2, 16, 128, seed=11, prefix=prefix)
    nq = 3
    q = _q(2, 8, nq, 128, 12)
    clean_o, clean_l = _call(c, q)
    for b, n in enumerate(c.lens):
        p = int(c.tables[b, (n - 1) // 16])
        c.k[p, :, (n - 1) % 16] = math.nan
        c.v[p, :, (n - 1) % 16] = math.inf
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.equal(o[:, :, :nq - 1], clean_o[:, :, :nq - 1]) and torch.equal(lse[:, :, :nq - 1], clean_l[:, :, :nq - 1])
    assert torch.isnan(lse[:, :, nq - 1]).all()


@pytest.mark.parametrize("B,g,nq,prefix", [(3, 1, 5, 0), (3, 2, 7, 0), (3, 4, 8, 0), (3, 3, 20, 0), (3, 1, 5, 100), (30, 1, 5, 700)])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_newer_tokens_may_hold_anything(B, g, nq, prefix, d):
    """Infinities and NaN in single values of the last new tokens: rows that do not see those tokens stay as they
    are, bit by bit; rows that do get what a sum with such a term gives, in that column only."""
    lens = [150, 64 + nq, 3 * nq] + [90] * (B - 3)
    c = Cache(lens, 2, 16, d, seed=nq + d, prefix=prefix)
    q = _q(B, 2 * g, nq, d, 12)
    clean_o, clean_l = _call(c, q)
    check_decode(c, q, clean_o, clean_l, 1 / math.sqrt(d), seqs=[0, 1, 2])
    bad = {nq // 2: (3, math.inf), nq - 1: (d - 2, math.nan)}  # new token: column, value
    for b, n in enumerate(lens):
        for i, (col, x) in bad.items():
            j = n - nq + i
            c.v[int(c.tables[b, j // 16]), :, j % 16, col] = x
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.equal(lse, clean_l)
    for i in range(nq):
        same = torch.ones(d, dtype=torch.bool)
        for first, (col, x) in bad.items():
            if i >= first:
                same[col] = False
                got = o[:, :, i, col]
                assert bool((torch.isnan(got) if math.isnan(x) else torch.isnan(got) | (got == x)).all()), (i, col)
        assert torch.equal(o[:, :, i, same], clean_o[:, :, i, same]), i


@pytest.mark.parametrize("prefix", [0, 333, 5000])
def test_strided_queries_and_outputs(prefix):
    """Token-major views of queries and outputs; what lies between the rows of the output stays."""
    B, hq, nq, d = 5, 8, 2, 64
    c = Cache((100, 3, 0, 64, 257), 2, 16, d, seed=13, prefix=prefix, rows_first=True, one_tensor=True)
    big = torch.randn((B, nq, 2 * hq, d), generator=torch.Generator().manual_seed(14)).to(torch.bfloat16).cuda()
    q = big[:, :, :hq].transpose(1, 2)
    store = torch.full((B, nq, 2 * hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    out = store[:, :, hq:].transpose(1, 2)
    lse = torch.empty((B, hq, nq), dtype=torch.float32, device="cuda")
    o, l = _call(c, q, out=out, lse=lse)
    assert o is out and l is lse and fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / 8)
    assert (store[:, :, :hq] == 5.0).all()


@pytest.mark.parametrize("prefix", [0, 40, 4000])
def test_scratch_of_any_contents_and_equal_results(prefix):
    B, hq, nq, d = 30, 8, 1, 128
    rng = np.random.default_rng(15)
    c = Cache(rng.integers(0, 900, B).tolist(), 2, 16, d, seed=15, prefix=prefix)
    q = _q(B, hq, nq, d, 16)
    n = fa.fa_decode_shared_workspace_bytes(B, hq, 2, nq, prefix, d)
    assert n >= fa.fa_decode_paged_workspace_bytes(B, hq, 2, nq, d) > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    o0, l0 = _call(c, q, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o0, l0, 1 / math.sqrt(d))
    for fill in (0, 127, 255):
        ws.fill_(fill)
        o, l = _call(c, q, workspace=ws)
        assert torch.equal(o, o0) and torch.equal(l, l0)
    with pytest.raises(fa.FAError):
        _call(c, q, workspace=ws[:n - 256])


@pytest.mark.parametrize("prefix", [0, 500])
@pytest.mark.parametrize("break_it", ["page", "page_high", "length", "negative"])
def test_bad_contents_are_reported(break_it, prefix):
    """The wrong sequence is reported and its neighbours' rows are right."""
    c = Cache((90, 70, 33), 2, 16, 64, seed=17, prefix=prefix)
    q = _q(3, 4, 1, 64, 18)
    tables, lens = c.tables, c.seq_lens
    c.tables, c.seq_lens = tables.clone(), lens.clone()
    if break_it == "page":
        c.tables[1, 2] = -3
    elif break_it == "page_high":
        c.tables[1, 2] = 1 << 30
    elif break_it == "length":
        c.seq_lens[1] = 16 * tables.shape[1] + 1
    else:
        c.seq_lens[1] = -1
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert fa.fa_check_device_status() == fa.FA_OK
    c.tables, c.seq_lens = tables, lens
    check_decode(c, q, o, lse, 1 / 8, seqs=(0, 2))


def test_bad_prefix_page_is_reported():
    c = Cache((9, 7), 2, 16, 64, seed=19, prefix=100)
    q = _q(2, 4, 1, 64, 20)
    good = c.prefix_pages.clone()
    c.prefix_pages[3] = c.pages
    _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    c.prefix_pages = good
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o, lse, 1 / 8)


@pytest.mark.parametrize("prefix", [0, 300, 2000])
def test_captured_call_follows_lengths_and_tables(prefix):
    B, hq, d = 24, 8, 64
    full = [200] * B
    c = Cache(full, 2, 16, d, seed=21, prefix=prefix)
    q = _q(B, hq, 1, d, 22)
    _call(c, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = _call(c, q)
    rng = np.random.default_rng(23)
    for step in range(3):
        c.lens = [0] * B if step == 1 else rng.integers(0, 201, B).tolist()
        c.seq_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.tables.copy_(c.tables[torch.randperm(B, device="cuda")].clone())
        q.copy_(_q(B, hq, 1, d, 24 + step))
        graph.replay()
        assert fa.fa_check_device_status() == fa.FA_OK
        check_decode(c, q, o, lse, 1 / 8)


@pytest.mark.parametrize("prefix", [0, 300, 2000])
def test_two_streams_at_once(prefix):
    """Calls in flight on two streams, each with its own scratch."""
    c = Cache((3000, 500, 40) * 8, 2, 16, 128, seed=25, prefix=prefix)
    qs = [_q(24, 8, 1, 128, 26 + i) for i in range(2)]
    want = [_call(c, q) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_call(c, qs[i]))
    torch.cuda.synchronize()
    assert fa.fa_check_device_status() == fa.FA_OK
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_default_stream_scratch_is_shared_by_calls_of_all_sizes():
    """Calls of different sizes and kinds, one after another on the default stream, and from two threads at once."""
    import threading
    cases = [Cache((900, 30), 2, 16, 128, seed=40), Cache((2000,) * 6, 4, 16, 64, seed=41, prefix=300),
             Cache((5, 0, 9), 1, 16, 128, seed=42), Cache((100,) * 40, 2, 16, 64, seed=43, prefix=2500)]
    qs = [_q(len(c.lens), 8, 1, c.d, 44 + i) for i, c in enumerate(cases)]
    first = [_call(c, q) for c, q in zip(cases, qs)]
    for c, q, (o, l) in zip(cases, qs, first):
        check_decode(c, q, o, l, 1 / math.sqrt(c.d))
    got, errors = {}, []

    def work(k):
        try:
            got[k] = [[_call(c, q) for c, q in zip(cases, qs)] for _ in range(20)]
        except Exception as e:  # pragma: no cover
            errors.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors and fa.fa_check_device_status() == fa.FA_OK
    for k in got:
        for round_ in got[k]:
            for (o, l), (o0, l0) in zip(round_, first):
                assert torch.equal(o, o0) and torch.equal(l, l0)


def test_first_cuda_call_of_a_thread():
    """A thread that has made no CUDA call yet, on tensors and scratch that are there already."""
    import threading
    c = Cache((90, 3), 2, 16, 64, seed=45)
    q = _q(2, 4, 1, 64, 46)
    out, lse = torch.empty_like(q), torch.empty((2, 4, 1), device="cuda")
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(2, 4, 2, 1, 64), dtype=torch.uint8, device="cuda")
    k = torch.randn((1, 1, 64, 64), device="cuda").to(torch.bfloat16)
    o, l = torch.empty_like(k), torch.empty((1, 1, 64), device="cuda")
    torch.cuda.synchronize()
    codes = []

    def first(fn):
        try:
            fn()
            codes.append(fa.FA_OK)
        except fa.FAError as e:
            codes.append(e.code)
    for fn in (lambda: fa.fa_decode_paged(q, c.k, c.v, c.tables, c.seq_lens, 0.125, out, lse, ws),
               lambda: fa.fa_fwd(k, k, k, 0.125, out=o, lse=l)):
        t = threading.Thread(target=first, args=(fn,))
        t.start()
        t.join()
    assert codes == [fa.FA_OK, fa.FA_OK] and fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, out, lse, 0.125)


def test_pool_offsets_beyond_32_bits():
    page, hkv, d = 256, 8, 128
    pages = (1 << 32) // (page * hkv * d) + 4
    k = torch.empty((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Cache((700,), hkv, page, d, seed=27, prefix=300, spare=0)
    ids = torch.arange(pages - c.pages, pages, device="cuda")
    k[ids], v[ids] = c.k, c.v
    c.tables += pages - c.pages
    c.prefix_pages += pages - c.pages
    c.k, c.v = k, v
    _run(c, 8, 1, seed=28)
    c.prefix = 0
    _run(c, 8, 1, seed=29)


def test_same_page_named_twice():
    """A table may name a page more than once; a prefix page may also be an own page."""
    c = Cache((64, 48), 2, 16, 64, seed=30, prefix=32)
    c.tables[1, 1] = c.tables[0, 0]
    c.tables[0, 2] = c.tables[0, 1]
    c.tables[1, 2] = c.prefix_pages[0]
    _run(c, 4, 1, seed=31)


@pytest.mark.parametrize("lens,g,prefix", [([9000, 40], 1, 0), ([3000] * 12, 8, 0), ([300] * 20, 4, 2000), ([200, 100], 4, 900)])
def test_an_infinite_value_stays_infinite(lens, g, prefix):
    """One infinite value among equal scores makes its column infinite, not NaN, whatever parts the row is merged of."""
    c = Cache(lens, 2, 16, 128, seed=21, prefix=prefix)
    q = torch.zeros((len(lens), 2 * g, 1, 128), dtype=torch.bfloat16, device="cuda")
    for b, n in enumerate(lens):
        c.v[int(c.tables[b, n // 2 // 16]), :, n // 2 % 16, 5] = -math.inf
    o, lse = _call(c, q)
    assert fa.fa_check_device_status() == fa.FA_OK
    assert bool((o[..., 5] == -math.inf).all())
    assert bool(torch.isfinite(o[..., :5]).all()) and bool(torch.isfinite(o[..., 6:]).all()) and bool(torch.isfinite(lse).all())



def test_matches_the_dense_decode():
    B, H, nq, nk, d = 2, 3, 4, 500, 128
    c = Cache((nk,) * B, H, 16, d, seed=32)
    dense = lambda pool: torch.stack([pool[c.tables[b].long()].transpose(0, 1).reshape(H, -1, d)[:, :nk] for b in range(B)]).contiguous()
    q = _q(B, H * nq, 1, d, 33)
    o, lse = fa.fa_decode_paged(q, c.k, c.v, c.tables, c.seq_lens)
    od, ld = fa.fa_decode(q.view(B, H, nq, d), dense(c.k), dense(c.v))
    # both within half a bf16 step (output) plus half a step of P of the same value, LSE in fp32
    assert (o.view_as(od).double() - od.double()).abs().max() <= 4 * 2.0 ** -8 * float(od.abs().max())
    assert (lse.view_as(ld) - ld).abs().max() <= 1e-4


def test_refusals_with_tensors_on_the_gpu():
    c = Cache((20, 5), 2, 16, 64, seed=34, prefix=20)
    q = _q(2, 4, 1, 64, 35)
    a = dict(q=q, k_pages=c.k, v_pages=c.v, block_tables=c.tables, seq_lens=c.seq_lens)
    for kw in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[0]), dict(k_pages=c.k[:, :1]),
               dict(seq_lens=c.seq_lens[:1]), dict(block_tables=c.tables.long()), dict(out=q.float()),
               dict(out=q[:, :2]), dict(lse=torch.zeros(2, 4, device="cuda")), dict(q=q.cpu()),
               dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            fa.fa_decode_paged(**{**a, **kw})
    with pytest.raises(fa.FAError):
        fa.fa_decode_paged(**{**a, "q": q.expand(2, 4, 33, 64).contiguous()})  # 66 rows of a head
    with pytest.raises(fa.FAError):
        fa.fa_decode_paged(**{**a, "workspace": torch.zeros(8, dtype=torch.uint8, device="cuda")})
    with pytest.raises(ValueError):  # two pages hold 32 keys
        fa.fa_decode_shared(q, c.k, c.v, c.prefix_pages, 33, c.tables, c.seq_lens)


def test_a_serving_run():
    """Prompts appended at once, then steps of one token appended and attended to, against the packed causal
    forward over the same tokens; then the prompts' common start moved into a shared prefix."""
    hq, hkv, d, page, steps = 8, 2, 64, 16, 4
    common, prompts = 48, [70, 49, 130]
    B = len(prompts)
    g = torch.Generator().manual_seed(36)
    cos, sin = fa.fa_rope_tables(256, d, device="cuda")
    lens = [n + steps for n in prompts]
    x = [torch.randn((n, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).cuda() for n in lens]
    for t in x[1:]:
        t[:common] = x[0][:common]
    need = [-(-n // page) for n in lens]
    pool = torch.zeros((sum(need) + 8, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    k_pages, v_pages = pool, torch.zeros_like(pool)
    tables = torch.zeros((B, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    tables = tables.cuda()
    split = lambda t: (t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    # the prompts
    q, k, v = split(torch.cat([t[:n] for t, n in zip(x, prompts)]))
    cu = i32(np.concatenate([[0], np.cumsum(prompts)]).tolist())
    fa.fa_kv_append(k, v, k_pages, v_pages, tables, i32(prompts), cu, q=q, cos=cos, sin=sin)
    outs, shared_outs = [], []
    k2, v2 = k_pages.clone(), v_pages.clone()
    for s in range(steps):
        seq = i32([n + s + 1 for n in prompts])
        q, k, v = split(torch.stack([t[n + s] for t, n in zip(x, prompts)]))
        qr = fa.fa_kv_append(k, v, k_pages, v_pages, tables, seq, q=q, cos=cos, sin=sin)
        outs.append(fa.fa_decode_paged(qr.unsqueeze(2), k_pages, v_pages, tables, seq)[0])
        # the first three pages of sequence 0 are everybody's prefix; own keys are appended behind them
        own = seq - common
        pos = i32([n + s for n in prompts])
        qr = fa.fa_kv_append(k, v, k2, v2, tables[:, common // page:].contiguous(), own, q=q, cos=cos, sin=sin, positions=pos)
        shared_outs.append(fa.fa_decode_shared(qr.unsqueeze(2), k2, v2, tables[0, :common // page].contiguous(), common,
                                               tables[:, common // page:].contiguous(), own)[0])
    assert fa.fa_check_device_status() == fa.FA_OK
    assert torch.equal(k_pages, k2) and torch.equal(v_pages, v2)
    # the same tokens through the packed causal forward, K/V heads repeated for their group
    cu_all = i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    q, k, v = split(torch.cat(x))
    scratch_k, scratch_v = torch.zeros_like(pool), torch.zeros_like(pool)
    qr = fa.fa_kv_append(k, v, scratch_k, scratch_v, tables, i32(lens), cu_all, q=q, cos=cos, sin=sin)
    rows = lambda pages, b: pages[tables[b].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :lens[b]].transpose(0, 1)
    kr = torch.cat([rows(scratch_k, b) for b in range(B)]).repeat_interleave(hq // hkv, 1).contiguous()
    vr = torch.cat([rows(scratch_v, b) for b in range(B)]).repeat_interleave(hq // hkv, 1).contiguous()
    ref, _ = fa.fa_fwd_varlen(qr, kr, vr, cu_all, max(lens), causal=True)
    start = np.concatenate([[0], np.cumsum(lens)])
    for s in range(steps):
        want = torch.stack([ref[start[b] + prompts[b] + s] for b in range(B)]).double()
        # two roundings of half a bf16 step on each side, of weights and output, relative to the largest output
        tol = 4 * 2.0 ** -8 * float(want.abs().max())
        assert (outs[s].squeeze(2).double() - want).abs().max() <= tol
        assert (shared_outs[s].squeeze(2).double() - want).abs().max() <= tol
