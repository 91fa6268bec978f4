"""Prompt operators and eviction on tensors of more than 2^31 elements: offsets past 32 bits, at the far end."""
import math

import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache
from prompt_utils import Paged, Prompts, bf16_randn, check_backward, check_forward, check_weights, offsets

pytestmark = pytest.mark.gpu

FRONT = 131100  # tokens before the first sequence: 131100 * 128 heads * 128 > 2^31


class Far(Prompts):
    """Sequences at the end of tensors that hold NaN before them."""

    def __init__(self, n, hq, hkv, d, seed):
        self.n = self.m = list(n)
        self.hq, self.hkv, self.d, self.g, self.pad = hq, hkv, d, hq // hkv, (FRONT, 0)
        live = sum(n)
        self.total = self.total_k = FRONT + live

        def tensor(heads, s):
            x = torch.full((self.total, heads, d), math.nan, dtype=torch.bfloat16, device="cuda")
            x[FRONT:] = bf16_randn((live, heads, d), s)
            return x

        self.q, self.do, self.k, self.v = tensor(hq, seed), tensor(hq, seed + 1), tensor(hkv, seed + 2), tensor(hkv, seed + 3)
        self.cu_q = self.cu_k = offsets(self.n, FRONT)
        self.max_q = self.max_k = max(n)


@pytest.mark.parametrize("hkv", [128, 4])
def test_packed(hkv):
    c = Far((70, 3), 128, hkv, 128, seed=hkv)
    scale = 1 / math.sqrt(128)
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, c.max_q)
    check_forward(c, o, lse, scale)
    w = torch.zeros((2, hkv, 75), device="cuda")
    fa.fa_prompt_key_weights(c.q, c.k, lse, w, c.cu_q, c.max_q, accumulate=False)
    check_weights(c, w, torch.zeros_like(w), lse, scale, accumulate=False)
    check_backward(c, *fa.fa_prompt_bwd(c.q, c.k, c.v, o, c.do, lse, c.cu_q, c.max_q), scale)
    assert fa.fa_check_device_status() == fa.FA_OK


def test_pages():
    """A pool of 2.2e9 elements whose last pages are used."""
    cache = Cache((500, 129), 8, 128, 128, seed=1, spare=8)
    far = 16800  # 16800 pages of 8 heads of 128 rows of 128
    for name in ("k", "v"):
        big = torch.full((far + cache.pages, 8, 128, 128), math.nan, dtype=torch.bfloat16, device="cuda")
        big[far:] = getattr(cache, name)
        setattr(cache, name, big)
    cache.tables = torch.where(cache.tables >= 0, cache.tables + far, cache.tables)
    spare = torch.tensor(sorted(set(range(cache.pages)) - cache.used), dtype=torch.int32) + far
    cache.pages += far
    c = Paged((60, 129), cache, 16, seed=2)
    scale = 1 / math.sqrt(128)
    o, lse = fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, c.cu_q, 129)
    check_forward(c, o, lse, scale)
    w = torch.zeros((2, 8, 500), device="cuda")
    fa.fa_prompt_key_weights_paged(c.q, cache.k, cache.tables, cache.seq_lens, lse, w, c.cu_q, 129, accumulate=False)
    check_weights(c, w, torch.zeros_like(w), lse, scale, accumulate=False)
    k0, v0 = ([x[cache.tables[0, :4].long()].transpose(0, 1).reshape(8, -1, 128).clone() for x in (cache.k, cache.v)])
    new = spare[:4].view(2, 2).cuda()
    new_w = torch.zeros((2, 8, 200), device="cuda")
    lens, kept = fa.fa_kv_evict(cache.k, cache.v, cache.tables, cache.seq_lens, w, 200, 20, new_tables=new, new_weights=new_w)
    assert lens.tolist() == [200, 129]
    for x, old in ((cache.k, k0), (cache.v, v0)):
        got = x[new[0].long()].transpose(0, 1).reshape(8, -1, 128)[:, :200]
        want = torch.stack([old[h, kept[0, h].long()] for h in range(8)])
        assert torch.equal(got, want)
    assert fa.fa_check_device_status() == fa.FA_OK
