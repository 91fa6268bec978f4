"""Blocks that one CTA works at for longer than a second: no warp gives up waiting for another."""
import math

import pytest
import torch

import exact_attention_30_gb300 as fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_forward_over_one_range_of_keys(d):
    """One token over 2^29 keys, not cut into ranges (no workspace): all but the last page are one page, of score 0 and
    values +-1; the last one's keys have score 16 and value 2, so that LSE and O need every tile."""
    keys, page = 1 << 29, 1024
    k, v = (torch.zeros((2, 1, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[1, :, :, 0] = 4
    v[0, :, 0::2], v[0, :, 1::2], v[1] = 1, -1, 2
    q = torch.zeros((1, 1, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 4
    tables = torch.zeros((1, keys // page), dtype=torch.int32, device="cuda")
    tables[0, -1] = 1
    lens, cu = torch.tensor([keys], dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda()
    o, lse = fa.fa_prompt_paged(q, k, v, tables, lens, cu, 1, scale=1.0,
                                workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert fa.fa_check_device_status() == fa.FA_OK
    top = page * math.exp(16)
    total = top + keys - page
    # half a step of bf16 for O and for the weights; the sums of the weights are in steps of 128 up to 2^29, exact
    assert (o.double() - 2 * top / total).abs().max().item() <= 2 * 2.0 ** -8 * 2 * top / total
    assert abs(lse.item() - math.log(total)) <= 2.0 ** -18 * math.log(total)


def test_weights_of_the_first_keys_of_a_long_prompt():
    """1.25 million tokens of 128 heads: the first unit meets as many query tiles. Scores are 0 and LSE_i = ln(i + 1), so
    w_j = 128 sum over i >= j of 1 / (i + 1)."""
    n, hq, d = 1_250_000, 128, 64
    q = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(1, n + 1, dtype=torch.float64, device="cuda")
    lse = at.log().float().expand(hq, n).contiguous()
    w = torch.zeros((1, 1, n), device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    fa.fa_prompt_key_weights(q, k, lse, w, cu, n)
    assert fa.fa_check_device_status() == fa.FA_OK
    p = torch.exp(-lse[0].double())
    ref = hq * p.flip(0).cumsum(0).flip(0)
    # rounding -LSE * log2(e) moves the exponent by up to 2^-24 * 20.3, the exponential adds 2^-22, the sums 2^-20
    err = ((w[0, 0].double() - ref).abs() / ref).max().item()
    assert err <= 2.0 ** -18, err


def test_workspace_of_tables_past_the_longest_sequence():
    """max_pages * page_size past 2^30 keys plans as 2^30 do, which is what fa_prompt_paged takes of such a table."""
    for b, hq, hkv, t, d in ((1, 8, 2, 60, 128), (3, 4, 4, 1, 64)):
        n = fa.fa_prompt_fwd_workspace_bytes(b, hq, hkv, t, t, 1 << 30, d)
        assert n > 0
        for keys in ((1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 1):
            assert fa.fa_prompt_fwd_workspace_bytes(b, hq, hkv, t, t, keys, d) == n
