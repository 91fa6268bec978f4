"""fa_kv_evict against a plain selection and copy, and the operators of a cache that is cut back, in a run."""
import math

import numpy as np
import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache, to64
from prompt_utils import Prompts, attention64, bf16_randn, offsets

pytestmark = pytest.mark.gpu


def _stay(w, m, budget, recent):
    """Indices that stay of m weights."""
    c, old = min(m, budget), m - min(recent, m)
    key = [(-(math.inf if x != x else x), 0 if x != x else 1, j) for j, x in enumerate(w[:old])]
    best = sorted(range(old), key=lambda j: key[j])[:max(0, c - (m - old))]
    return sorted(best) + list(range(old, m))


def _rows(cache, pool, table, n, h):
    idx = [int(table[i // cache.page]) for i in range(n)]
    return torch.stack([pool[p, h, i % cache.page] for i, p in enumerate(idx)]) if n else pool[:0, h, 0]


def _check(cache, w, budget, recent, in_place, spare_pages=None):
    B, hkv = len(cache.lens), cache.hkv
    w0, k0, v0 = w.clone(), cache.k.clone(), cache.v.clone()
    if in_place:
        tables, new_w = cache.tables, w
        lens, kept = fa.fa_kv_evict(cache.k, cache.v, cache.tables, cache.seq_lens, w, budget, recent)
    else:
        tables, new_w = spare_pages, torch.full((B, hkv, budget + 2), 7.0, device="cuda")
        lens, kept = fa.fa_kv_evict(cache.k, cache.v, cache.tables, cache.seq_lens, w, budget, recent,
                                    new_tables=tables, new_weights=new_w)
        assert torch.equal(w.view(torch.int32), w0.view(torch.int32))
    assert fa.fa_check_device_status() == fa.FA_OK
    assert lens.tolist() == [min(m, budget) for m in cache.lens]
    old_t, new_t, wl = cache.tables.cpu(), tables.cpu(), w0.cpu().numpy().astype(np.float32)
    for b, m in enumerate(cache.lens):
        c = min(m, budget)
        for h in range(hkv):
            stay = _stay(wl[b, h].tolist(), m, budget, recent)
            assert kept[b, h, :c].tolist() == stay and (kept[b, h, c:] == -1).all(), (b, h)
            st = torch.tensor(stay, dtype=torch.long)
            got_w = new_w[b, h, :c].cpu()
            assert torch.equal(got_w.nan_to_num(nan=-5.0), w0[b, h].cpu()[st].nan_to_num(nan=-5.0))
            if not in_place:
                assert (new_w[b, h, c:] == 7).all()
            for new, old in ((cache.k, k0), (cache.v, v0)):
                want = _rows(cache, old, old_t[b], m, h)[st]
                assert torch.equal(_rows(cache, new, new_t[b], c, h), want), (b, h)


def _spare_tables(cache, budget, extra):
    """Pages at the pool's end, one sequence after the other."""
    need = [-(-min(m, budget) // cache.page) for m in cache.lens]
    assert sum(need) <= extra
    t = torch.full((len(need), max([1] + need + [-(-min(budget, cache.tables.shape[1] * cache.page) // cache.page)])), -9,
                   dtype=torch.int32)
    free = sorted(set(range(cache.pages)) - cache.used)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(free[:n], dtype=torch.int32)
        free = free[n:]
    return t.cuda()


def _weights(shape, seed, kind):
    g = torch.Generator().manual_seed(seed)
    w = (2 * torch.randn(shape, generator=g)).exp()
    if kind == "ties":
        w = (w * 2).floor().clamp(max=3)
    elif kind == "zero":
        w.zero_()
    elif kind == "odd":
        w = torch.randn(shape, generator=g)
        r = torch.rand(shape, generator=g)
        w[r < 0.1], w[(r > 0.1) & (r < 0.2)], w[(r > 0.2) & (r < 0.25)] = 0.0, -0.0, math.inf
        w[(r > 0.25) & (r < 0.3)], w[(r > 0.3) & (r < 0.35)] = -math.inf, math.nan
    return w.cuda()


@pytest.mark.parametrize("page", [8, 24, 64, 1000])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 0), (64, 16), (100, 100), (257, 1), (5000, 10)])
@pytest.mark.parametrize("in_place", [True, False])
def test_lengths_budgets_and_pages(page, budget, recent, in_place):
    lens = (0, 1, 2, 63, 64, 65, 100, 101, 257, 700)
    extra = sum(-(-min(m, budget) // page) for m in lens) + 2
    cache = Cache(lens, 2, page, 128 if budget % 2 else 64, seed=page, rows_first=budget > 64, spare=extra)
    w = _weights((len(lens), 2, 705), budget, "plain")
    _check(cache, w, budget, recent, in_place, None if in_place else _spare_tables(cache, budget, extra))


@pytest.mark.parametrize("kind", ["ties", "zero", "odd"])
@pytest.mark.parametrize("in_place", [True, False])
def test_equal_and_odd_weights(kind, in_place):
    lens = (1500, 90, 33)
    extra = 20
    cache = Cache(lens, 3, 64, 64, seed=1, spare=extra)
    w = _weights((3, 3, 1500), 2, kind)
    _check(cache, w, 300, 40, in_place, None if in_place else _spare_tables(cache, 300, extra))


def test_long_sequences_in_place():
    """Many batches of rows and chunks of weights; keys and values side by side in one tensor."""
    cache = Cache((9000, 12345), 2, 16, 128, seed=3, one_tensor=True)
    _check(cache, _weights((2, 2, 13000), 4, "plain"), 7001, 50, True)


@pytest.mark.parametrize("kind", ["plain", "ties"])
@pytest.mark.parametrize("in_place", [True, False])
def test_weights_past_shared_memory(kind, in_place):
    """65000 weights and indices do not fit: the weights are read again for each step of the selection."""
    extra = 160
    cache = Cache((60000, 50001, 17), 1, 64, 64, seed=4, spare=extra)
    w = _weights((3, 1, 60000), 5, kind)
    _check(cache, w, 5000, 100, in_place, None if in_place else _spare_tables(cache, 5000, extra))


def test_no_row_moves_when_all_stay():
    cache = Cache((100, 40), 1, 16, 64, seed=5)
    _check(cache, _weights((2, 1, 100), 6, "plain"), 100, 0, True)


def test_step_by_step_in_place_in_a_graph():
    """One more key, one key out, lengths and weights in place: the same as the plain form step by step."""
    cache = Cache((65, 65), 2, 16, 64, seed=7, width_extra=1)
    lens = cache.seq_lens.clone()
    w = _weights((2, 2, 65), 8, "plain")
    kept = torch.empty((2, 2, 64), dtype=torch.int32, device="cuda")
    run = lambda: fa.fa_kv_evict(cache.k, cache.v, cache.tables, lens, w, 64, 8, new_lens=lens, kept=kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = [t.clone() for t in (cache.k, cache.v, lens, w)]
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t, s in zip((cache.k, cache.v, lens, w), saved):
        t.copy_(s)
    for step in range(5):
        lens.fill_(65)
        w[:, :, 64] = float(step)
        before = w.clone(), cache.k.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [64, 64]
        for b in range(2):
            for h in range(2):
                stay = _stay(before[0][b, h].tolist(), 65, 64, 8)
                assert kept[b, h].tolist() == stay
                want = _rows(cache, before[1], cache.tables[b].cpu(), 65, h)[torch.tensor(stay)]
                assert torch.equal(_rows(cache, cache.k, cache.tables[b].cpu(), 64, h), want)


def test_bad_lengths_and_pages():
    for bad in (-1, 1000):
        cache = Cache((200, 90), 2, 16, 64, seed=4)
        lens = torch.tensor([bad, 90], dtype=torch.int32).cuda()
        k0 = cache.k.clone()
        new_lens, kept = fa.fa_kv_evict(cache.k, cache.v, cache.tables, lens, _weights((2, 2, 300), 1, "plain"), 50, 5)
        assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
        assert new_lens.tolist() == [bad, 50] and (kept[0] == -1).all() and (kept[1] >= 0).all()
        mine = [int(p) for p in cache.tables[0, :13]]
        assert torch.equal(cache.k[mine], k0[mine])
    cache = Cache((200, 90), 2, 16, 64, seed=4)
    cache.tables[0, 12] = 1 << 30
    fa.fa_kv_evict(cache.k, cache.v, cache.tables, cache.seq_lens, _weights((2, 2, 300), 1, "plain"), 50, 5)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG


def test_refusals():
    cache = Cache((200, 90), 2, 16, 64, seed=4)
    w = torch.zeros((2, 2, 200), device="cuda")
    call = lambda **kw: fa.fa_kv_evict(**{**dict(k_pages=cache.k, v_pages=cache.v, block_tables=cache.tables,
                                                 seq_lens=cache.seq_lens, weights=w, budget=50), **kw})
    for kw in (dict(weights=w.half()), dict(new_tables=cache.tables[:1]), dict(new_weights=w[:, :, :49]),
               dict(new_lens=cache.seq_lens.long()), dict(kept=torch.zeros((2, 2, 51), dtype=torch.int32, device="cuda")),
               dict(budget=1 << 40)):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(budget=0), dict(recent=-1), dict(recent=51), dict(new_tables=cache.tables[:, :3].contiguous())):
        with pytest.raises(fa.FAError):
            call(**kw)


def test_prompt_weights_eviction_and_decoding_in_a_run():
    """A prompt's attention and key weights, its cache cut back, then steps that append, attend and add weights, and a
    second turn of several tokens over what is left: every attention against fp64 over the keys that stayed."""
    hq, hkv, d, page, budget, recent = 8, 2, 64, 16, 48, 8
    n = [130, 75]
    c = Prompts(n, hq, hkv, d, seed=21)
    scale = 1 / 8
    pages = 40
    k_pages = torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v_pages = torch.zeros_like(k_pages)
    tables = torch.randperm(pages, generator=torch.Generator().manual_seed(3))[:24].reshape(2, 12).to(torch.int32).cuda()
    lens = torch.tensor(n, dtype=torch.int32).cuda()
    cos, sin = fa.fa_rope_tables(400, d, device="cuda")
    q = fa.fa_kv_append(c.k, c.v, k_pages, v_pages, tables, lens, c.cu_q, q=c.q, cos=cos, sin=sin)
    o, lse = fa.fa_prompt_paged(q, k_pages, v_pages, tables, lens, c.cu_q, max(n))
    w = torch.zeros((2, hkv, 12 * page), device="cuda")
    fa.fa_prompt_key_weights_paged(q, k_pages, tables, lens, lse, w, c.cu_q, max(n))

    keys = lambda pool, b, h, m: torch.stack([pool[int(tables[b, i // page]), h, i % page] for i in range(m)]).cpu().double()

    def check(q3, o3, cu):  # tokens of sequence b in packed order, over its keys as they are in the cache
        for b in range(2):
            m, rows = int(lens[b]), slice(int(cu[b]), int(cu[b + 1]))
            for h in range(hkv):
                hs = slice(h * 4, h * 4 + 4)
                k, v = keys(k_pages, b, h, m), keys(v_pages, b, h, m)
                ref, _, p = attention64(q3[rows, hs].transpose(0, 1).cpu().double(), k, v, scale)
                got = o3[rows, hs].transpose(0, 1).cpu().double()
                # a rounding of each weight and of the sum, and 2^-12 for the scores
                assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * (p @ v.abs())).all()

    check(q, o, c.cu_q)
    model = [[w[b, h, :n[b]].cpu().double() for h in range(hkv)] for b in range(2)]
    total = list(n)  # tokens seen: the rotary positions go on
    for step in range(4):
        if step % 2 == 0:
            _, kept = fa.fa_kv_evict(k_pages, v_pages, tables, lens, w, budget, recent, new_lens=lens)
            for b in range(2):
                for h in range(hkv):
                    stay = _stay(model[b][h].float().tolist(), len(model[b][h]), budget, recent)
                    assert kept[b, h, :len(stay)].tolist() == stay
                    model[b][h] = model[b][h][torch.tensor(stay)]
            assert lens.tolist() == [budget, budget]
        new = 1 if step < 3 else 20
        cu = offsets((new, new))
        qkv = bf16_randn((2 * new, hq + 2 * hkv, d), 50 + step)
        pos = torch.tensor([t + i for t in total for i in range(new)], dtype=torch.int32).cuda()
        lens += new
        total = [t + new for t in total]
        q = fa.fa_kv_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], k_pages, v_pages, tables, lens, cu, q=qkv[:, :hq],
                            cos=cos, sin=sin, positions=pos)
        if new == 1:
            q4 = q.reshape(2, hq, 1, d)
            o, lse = fa.fa_decode_paged(q4, k_pages, v_pages, tables, lens)
            fa.fa_decode_key_weights(q4, k_pages, tables, lens, lse, w)
            check(q, o[:, :, 0], cu)
        else:
            o, lse = fa.fa_prompt_paged(q, k_pages, v_pages, tables, lens, cu, new)
            fa.fa_prompt_key_weights_paged(q, k_pages, tables, lens, lse, w, cu, new)
            check(q, o, cu)
        # the accumulated weights, in the kernels' fp32: what the next eviction goes by
        for b in range(2):
            for h in range(hkv):
                m = int(lens[b])
                got = w[b, h, :m].cpu().double()
                old = torch.cat([model[b][h], torch.zeros(new, dtype=torch.float64)])
                assert (got >= old - 1e-6 * (1 + old)).all()
                assert abs((got - old).sum().item() - 4 * new) <= 1e-4 * new
                model[b][h] = got
    assert fa.fa_check_device_status() == fa.FA_OK
