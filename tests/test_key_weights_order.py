"""The keys' weights are summed in a fixed order: the same bits whatever CTA takes a unit, and after which others."""
import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache
from prompt_utils import Paged, Prompts, check_weights, offsets

pytestmark = pytest.mark.gpu

LENS = (5000, 1700, 3100, 900, 4200, 301, 2500)


@pytest.mark.parametrize("hq,hkv,d,window", [(32, 8, 128, 0), (32, 8, 64, 0), (28, 4, 128, 0), (32, 8, 128, 700)])
def test_packed_repeats_itself(hq, hkv, d, window):
    """Several units to a CTA: twelve calls, and each sequence by itself, whose units are a CTA's first."""
    c = Prompts(LENS, hq, hkv, d, seed=hq + d)
    _, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, c.max_q)
    run = lambda: fa.fa_prompt_key_weights(c.q, c.k, lse, torch.zeros((len(LENS), hkv, max(LENS)), device="cuda"), c.cu_q,
                                           c.max_q, window=window)
    first = run()
    for _ in range(11):
        assert torch.equal(run(), first)
    for b, rows, _, n, _ in c.seqs():
        w = torch.zeros((1, hkv, max(LENS)), device="cuda")
        fa.fa_prompt_key_weights(c.q[rows], c.k[rows], lse[:, rows].contiguous(), w, offsets([n]), n, window=window)
        assert torch.equal(w[0], first[b]), b
    assert fa.fa_check_device_status() == fa.FA_OK


@pytest.mark.parametrize("width_extra", [0, 6000])
def test_paged_repeats_itself(width_extra):
    """Tables of the sequences' width, whose units CTAs take over, and far wider ones, whose list they go through in strides."""
    cache = Cache((6000, 2048, 3333, 4100), 8, 64, 128, seed=1, width_extra=width_extra)
    c = Paged((5000, 2048, 3000, 900), cache, 32, seed=2)
    _, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 5000)
    run = lambda: fa.fa_prompt_key_weights_paged(c.q, cache.k, cache.tables, cache.seq_lens, lse,
                                                 torch.zeros((4, 8, cache.tables.shape[1] * 64), device="cuda"), c.cu_q, 5000)
    first = run()
    for _ in range(11):
        assert torch.equal(run(), first)
    assert fa.fa_check_device_status() == fa.FA_OK


@pytest.mark.parametrize("width_extra", [0, 100])
def test_more_units_than_ctas(width_extra):
    """3712 units of 256 keys in full tables, several to a CTA index; some sequences have none."""
    lens = [300 if b % 30 else 0 for b in range(120)]
    cache = Cache(lens, 16, 64, 64, seed=5, width_extra=width_extra)
    cache.poison()
    c = Paged([3 if m else 0 for m in lens], cache, 16, seed=6)
    _, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 3)
    w = torch.rand((120, 16, cache.tables.shape[1] * 64), device="cuda")
    before = w.clone()
    fa.fa_prompt_key_weights_paged(c.q, cache.k, cache.tables, cache.seq_lens, lse, w, c.cu_q, 3)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_weights(c, w, before, lse, 1 / 8)


@pytest.mark.parametrize("n", [1, 40, 700, 3000])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_weights_stay_infinite(n, d):
    """Log-sum-exps that are too small by 200: e^200 is past fp32, for a prompt as for a step; keys that no counted
    token sees with such a one keep their weight."""
    c = Prompts((n, 65), 8, 2, d, seed=n)
    _, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, c.max_q)
    ref = fa.fa_prompt_key_weights(c.q, c.k, lse, torch.zeros((2, 2, max(n, 65)), device="cuda"), c.cu_q, c.max_q)
    tok = n // 2
    lse[:, tok] -= 200  # one token's: the keys up to it
    w = fa.fa_prompt_key_weights(c.q, c.k, lse, torch.zeros((2, 2, max(n, 65)), device="cuda"), c.cu_q, c.max_q)
    assert (w[0, :, :tok + 1] == float("inf")).all()
    assert torch.equal(w[0, :, tok + 1:], ref[0, :, tok + 1:]) and torch.equal(w[1], ref[1])


def test_infinite_weights_of_a_step():
    cache = Cache((700, 90), 2, 64, 128, seed=3)
    c = Paged((1, 1), cache, 8, seed=4)
    q = c.q[:, :, None].contiguous()
    _, lse = fa.fa_decode_paged(q, cache.k, cache.v, cache.tables, cache.seq_lens)
    lse[0] -= 200
    w = torch.zeros((2, 2, 700), device="cuda")
    fa.fa_decode_key_weights(q, cache.k, cache.tables, cache.seq_lens, lse, w, accumulate=False)
    v = torch.zeros_like(w)
    fa.fa_prompt_key_weights_paged(c.q, cache.k, cache.tables, cache.seq_lens, lse[..., 0].T.contiguous(), v, c.cu_q, 1,
                                   accumulate=False)
    assert (w[0] == float("inf")).all() and (v[0] == float("inf")).all()
    assert torch.isfinite(w[1]).all() and torch.isfinite(v[1]).all()
