"""Offsets out of order in fa_prompt_fwd and fa_prompt_paged: what is left out, and that nothing goes past its place."""
import math

import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache
from prompt_utils import Paged, Prompts, bf16_randn, check_forward

pytestmark = pytest.mark.gpu

BEHIND = 1 << 26  # bytes behind the workspace: more than any overrun of these sizes could reach


def _scratch(*sizes):
    n = fa.fa_prompt_fwd_workspace_bytes(*sizes)
    assert n > 0  # key ranges are planned
    return n, torch.full((n + BEHIND,), 7, dtype=torch.uint8, device="cuda")


def _untouched(out, lse, rows):
    keep = torch.ones(out.shape[0], dtype=torch.bool, device="cuda")
    for r in rows:
        keep[r] = False
    return bool((out[keep] == 3).all() and (lse[:, keep] == 3).all())


@pytest.mark.parametrize("hq,hkv,d,keys", [(4, 1, 128, 2000), (8, 2, 64, 700)])
def test_paged_back_and_forth(hq, hkv, d, keys):
    """A table far wider than the sequences: the kernel takes fewer key ranges than the host, and has more blocks."""
    cache = Cache((keys, keys, keys), hkv, 64, d, seed=1, width_extra=2000)
    q = bf16_randn((700, hq, d), 2)
    cu = torch.tensor([0, 640, 0, 640], dtype=torch.int32).cuda()
    n, ws = _scratch(3, hq, hkv, 700, 640, cache.tables.shape[1] * 64, d)
    out, lse = torch.full_like(q, 3.0), torch.full((hq, 700), 3.0, device="cuda")
    fa.fa_prompt_paged(q, cache.k, cache.v, cache.tables, cache.seq_lens, cu, 640, out=out, lse=lse, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert (ws[n:] == 7).all()
    assert _untouched(out, lse, [slice(0, 640)])


@pytest.mark.parametrize("b,t,hq,hkv,d", [(3, 1024, 1, 1, 64), (9, 1024, 8, 2, 128)])
def test_packed_back_and_forth(b, t, hq, hkv, d):
    c = Prompts((t,), hq, hkv, d, seed=b)
    cu = torch.tensor([0, t] * ((b + 1) // 2), dtype=torch.int32).cuda()
    n, ws = _scratch(b, hq, hkv, t, t, t, d)
    fa.fa_prompt_fwd(c.q, c.k, c.v, cu, t, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert (ws[n:] == 7).all()
    o, lse = fa.fa_prompt_fwd(c.q, c.k, c.v, c.cu_q, t, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_forward(c, o, lse, 1 / math.sqrt(d))


BAD = [([0, 90, 40, 150], []), ([0, 40, 151, 150], [0]), ([0, -1, 90, 150], [2])]  # offsets, the sequences that stay


@pytest.mark.parametrize("bad,stay", BAD)
@pytest.mark.parametrize("ranges", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_bad_offsets_are_left_out(bad, stay, ranges, d):
    """Others get what they get alone, whether keys are cut into ranges or not; rows of what is left out keep what they held."""
    cache = Cache((3000, 2000, 2500), 2, 64, d, seed=4)
    c = Paged((40, 50, 60), cache, 4, seed=9)
    cu = torch.tensor(bad, dtype=torch.int32).cuda()
    out, lse = torch.full_like(c.q, 3.0), torch.full((4, 150), 3.0, device="cuda")
    n = fa.fa_prompt_fwd_workspace_bytes(3, 4, 2, 150, 60, cache.tables.shape[1] * 64, d)
    assert n > 0
    ws = torch.empty(n if ranges else 0, dtype=torch.uint8, device="cuda")
    fa.fa_prompt_paged(c.q, cache.k, cache.v, cache.tables, cache.seq_lens, cu, 60, out=out, lse=lse, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert _untouched(out, lse, [slice(bad[b], bad[b + 1]) for b in stay])
    check_forward(c, out, lse, 1 / math.sqrt(d), seqs=stay)


@pytest.mark.parametrize("bad,stay", BAD)
def test_packed_bad_offsets_are_left_out(bad, stay):
    c = Prompts((40, 50, 60), 4, 2, 64, seed=9)
    cu = torch.tensor(bad, dtype=torch.int32).cuda()
    out, lse = torch.full_like(c.q, 3.0), torch.full((4, 150), 3.0, device="cuda")
    fa.fa_prompt_fwd(c.q, c.k, c.v, cu, 60, cu, 60, out=out, lse=lse)
    assert fa.fa_check_device_status() == fa.FA_ERR_INVALID_ARG
    assert _untouched(out, lse, [slice(bad[b], bad[b + 1]) for b in stay])
    check_forward(c, out, lse, 1 / 8, seqs=stay)
