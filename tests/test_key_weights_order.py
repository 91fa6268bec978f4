"""The keys' weights are summed in a fixed order: the same bits whatever CTA takes a unit, and after which others."""
import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache
from prompt_utils import Paged, Prompts, offsets

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
