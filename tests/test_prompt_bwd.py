"""fa_prompt_bwd on the GPU against the formulas in fp64, element by element, and against differences."""
import math

import pytest
import torch

import exact_attention_30_gb300 as fa
from prompt_utils import Prompts, attention64, bf16_randn, check_backward, offsets

pytestmark = pytest.mark.gpu

LENS = (0, 1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 200, 300)


def _grads(c, scale=None, **kw):
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, c.max_q, c.cu_k, c.max_k, scale=scale)
    g = fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, c.cu_q, c.max_q, c.cu_k, c.max_k, scale=scale, **kw)
    assert fa.fa_check_device_status() == fa.FA_OK
    return g


def _check(c, scale=None, **kw):
    g = _grads(c, scale, **kw)
    check_backward(c, *g, 1 / math.sqrt(c.d) if scale is None else scale)
    return g


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
    """Keys before the tokens; tokens without a key and keys without a token have gradients zero."""
    _check(Prompts((n, 17, n), 2 * g, 2, d, m=(m, 40, m), seed=n + m + g, pad=(1, 130)))


@pytest.mark.parametrize("lens,hq,hkv,d", [((1500, 700), 8, 2, 128), ((2100,), 5, 1, 64),
                                           ([(11 * i) % 70 for i in range(200)], 4, 2, 128)])
def test_many_units(lens, hq, hkv, d):
    """More key tiles than SMs: every CTA takes several, from the counter."""
    c = Prompts(lens, hq, hkv, d, seed=len(lens))
    g = _grads(c)
    check_backward(c, *g, 1 / math.sqrt(d), seqs=None if len(lens) < 5 else range(0, 200, 13))


def test_large_scores_and_scale():
    for scale in (0.5, 1.3):
        _check(Prompts((150, 260), 6, 2, 128, seed=3, big=16), scale)


def test_rows_outside_sequences_and_fused_gradients():
    c = Prompts((40, 0, 90), 8, 2, 64, seed=5, pad=(7, 9))
    grad = torch.full((c.total, 12, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = grad[:, :8], grad[:, 8:10], grad[:, 10:]
    got = _check(c, dq=dq, dk=dk, dv=dv)
    assert [t.data_ptr() for t in got] == [dq.data_ptr(), dk.data_ptr(), dv.data_ptr()]
    assert (grad[:7] == 5).all() and (grad[-9:] == 5).all()


@pytest.mark.parametrize("d", [64, 128])
def test_other_sequences_have_no_influence(d):
    """The next sequence's rows, not finite, stand in the last tiles of the one before."""
    c = Prompts((50, 70), 4, 1, d, seed=8)
    ref = _grads(c)
    for t in (c.k, c.v, c.q, c.do):
        t[50:] = math.nan
    c.v[60:] = math.inf
    got = _grads(c)
    for a, b in zip(got, ref):
        assert torch.equal(a[:50], b[:50])


def test_gradients_against_differences():
    """Sum of dO O along a random direction: central differences of the fp64 definition against the gradients'
    product with the direction. The bound is that of a sum of independent errors: each gradient element is off by
    some 2^-8 of its terms, and the sum of n of them by sqrt(n) of that; 8 such deviations."""
    c = Prompts((90, 33), 4, 2, 64, seed=11)
    dq, dk, dv = _grads(c)
    scale = 1 / 8
    g = torch.Generator().manual_seed(1)
    num = ana = var = 0.0
    for b, rows, keys, n, m in c.seqs():
        for h in range(2):
            q, k, v = c.head(b, rows, keys, h)
            hs = slice(2 * h, 2 * h + 2)
            do = c.do[rows, hs].transpose(0, 1).cpu().double()
            u = [torch.randn(x.shape, generator=g, dtype=torch.float64) for x in (q, k, v)]
            eps = 1e-5
            f = [(attention64(*(x + s * eps * y for x, y in zip((q, k, v), u)), scale)[0] * do).sum() for s in (1, -1)]
            num += (f[0] - f[1]).item() / (2 * eps)
            for y, t in zip(u, (dq[rows, hs].transpose(0, 1), dk[keys, h], dv[keys, h])):
                t = t.cpu().double()
                ana += (t * y).sum().item()
                var += (2.0 ** -8 * t.abs().max().item()) ** 2 * t.numel()
    assert abs(num - ana) <= 8 * math.sqrt(var), (num, ana, math.sqrt(var))


def test_graph_follows_offsets():
    c = Prompts((100, 28, 0), 8, 2, 128, seed=10)
    cu = c.cu_q.clone()
    o, lse = torch.zeros_like(c.q), torch.zeros((8, 128), device="cuda")
    out = [torch.zeros_like(t) for t in (c.q, c.k, c.v)]
    ws = torch.empty(fa.fa_prompt_bwd_workspace_bytes(3, 8, 2, 128, 128, 128, 128, 128), dtype=torch.uint8, device="cuda")

    def step():
        fa.fa_prompt_fwd(c.q, c.k, c.v, cu, 128, out=o, lse=lse)
        fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, cu, 128, dq=out[0], dk=out[1], dv=out[2], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ((100, 28, 0), (1, 1, 126), (0, 128, 0)):
        cu.copy_(offsets(lens))
        graph.replay()
        torch.cuda.synchronize()
        c.n = c.m = list(lens)
        check_backward(c, *out, 1 / math.sqrt(128))


def test_bad_offsets():
    c = Prompts((40, 50, 60), 4, 2, 64, seed=9)
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 60)
    cu = torch.tensor([0, 40, 151, 150], dtype=torch.int32).cuda()
    dq = torch.full_like(c.q, 3.0)
    g = fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, cu, 60, dq=dq)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    check_backward(c, *g, 1 / 8, seqs=[0])
    assert (dq[40:] == 3).all()


def test_no_tokens_or_no_keys():
    kv, e = bf16_randn((9, 2, 64), 1), torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    z, cu9 = torch.zeros(2, dtype=torch.int32).cuda(), offsets([9])
    lse = torch.empty((4, 0), device="cuda")
    dq, dk, dv = fa.fa_prompt_bwd(e, kv, kv, e, e, lse, z, 0, cu9, 9)
    assert dq.shape == e.shape and (dk == 0).all() and (dv == 0).all()
    q = bf16_randn((9, 4, 64), 2)
    o, lse = fa.fa_prompt_fwd(q, kv[:0], kv[:0], cu9, 9, z, 0)
    assert (o == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = fa.fa_prompt_bwd(q, kv[:0], kv[:0], o, q, lse, cu9, 9, z, 0)
    assert (dq == 0).all() and dk.shape == (0, 2, 64)
    assert fa.fa_check_device_status() == fa.FA_OK


def test_refusals():
    c = Prompts((8, 8), 4, 2, 64)
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 8)
    call = lambda **kw: fa.fa_prompt_bwd(**{**dict(q=c.q, k=c.k, v=c.v, o=o, do=c.do, lse=lse, cu_seqlens_q=c.cu_q,
                                                   max_seqlen_q=8), **kw})
    for kw in (dict(do=c.do.float()), dict(o=o[:8]), dict(lse=lse.T.contiguous()), dict(dk=torch.empty_like(c.q)),
               dict(workspace="x"), dict(dq=torch.empty((16, 4, 128), dtype=torch.bfloat16, device="cuda")[..., ::2])):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(max_seqlen_q=0), dict(scale=-1.0), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa.FAError):
            call(**kw)


def test_offsets_back_and_forth():
    """Sequences one upon another have more key tiles than the tokens: no partial sum goes past the workspace."""
    c = Prompts((512,), 4, 4, 64, seed=13)
    b = 9
    cu = torch.tensor([0, 512] * (b // 2 + 1), dtype=torch.int32).cuda()
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 512)
    n = fa.fa_prompt_bwd_workspace_bytes(b, 4, 4, 512, 512, 512, 512, 64)
    ws = torch.full((n + (1 << 22),), 7, dtype=torch.uint8, device="cuda")
    fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, cu, 512, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert (ws[n:] == 7).all()


def test_workspace_of_its_size_alone():
    """Few key tiles: their query ranges' partial sums lie inside the bytes asked for."""
    c = Prompts((300, 9, 77), 14, 2, 64, seed=15)
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, 300)
    n = fa.fa_prompt_bwd_workspace_bytes(3, 14, 2, c.total, c.total, 300, 300, 64)
    ws = torch.full((n + (1 << 22),), 255, dtype=torch.uint8, device="cuda")  # all NaN where anything were read unwritten
    g = fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, c.cu_q, 300, workspace=ws)
    check_backward(c, *g, 1 / 8)
    assert (ws[n:] == 255).all()
    again = fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, c.cu_q, 300, workspace=ws)
    assert torch.equal(again[1], g[1]) and torch.equal(again[2], g[2])  # a fixed order of sums
