"""The paged decode's abort path, driven without a fault.

fa_debug_decode_skip_load makes no CTA load the second tile of its walk (neither
the copies nor their expected bytes are issued), and a prefix's kernel load no
page at all. The consumers' bounded waits
run out, they free no stage any more, the producer stops by a bounded wait of
its own, waits for the copies it issued and ends; the merge reads whatever the
scratch then holds, within its bounds. The tests check that the timeout is
reported (and cleared by the read) and that ordinary calls on the same context,
with the same scratch, still match the fp64 definition.
"""
import ctypes
import math

import pytest
import torch

import exact_attention_30_gb300 as fa
from paged_utils import Cache, check_decode

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000  # 2 ms per bounded wait


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,g,nq,prefix", [
    ([24000, 300], 1, 1, 0),          # up to 8 rows; two or three tiles per CTA
    ([24000, 300], 4, 3, 0),          # 16
    ([24000, 300], 8, 3, 0),          # 32
    ([24000, 300], 8, 8, 0),          # 64
    ([14000, 0, 2500], 4, 1, 9000),   # the prefix as one more sequence
    ([2000] * 20, 4, 1, 30000),       # a prefix's kernel of 80 rows, the own keys beside it
    ([700] * 40, 8, 1, 30000),        # 320 rows: two query blocks
])
def test_skipped_tile_times_out_then_recovers(lens, g, nq, prefix, d):
    lib = fa.load_library()
    hkv = 2
    c = Cache(lens, hkv, 64, d, seed=d + g + nq, prefix=prefix)
    B, hq = len(lens), hkv * g
    gen = torch.Generator().manual_seed(7)
    q = torch.randn((B, hq, nq, d), generator=gen).to(torch.bfloat16).cuda()
    o = torch.empty_like(q)
    lse = torch.empty((B, hq, nq), dtype=torch.float32, device="cuda")
    n = fa.fa_decode_shared_workspace_bytes(B, hq, hkv, nq, prefix, d)
    ws = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
    scale = 1 / math.sqrt(d)
    pool = fa._pack_pool(c.k.data_ptr(), c.v.data_ptr(), c.pages, hkv, c.page, d, *c.k.stride()[:3], *c.v.stride()[:3])
    assert fa.fa_check_device_status() == fa.FA_OK
    rc = lib.fa_debug_decode_skip_load(
        q.data_ptr(), None, pool, c.prefix_pages.data_ptr() if prefix else None, prefix, c.tables.data_ptr(),
        c.tables.shape[1], c.seq_lens.data_ptr(), o.data_ptr(), None, lse.data_ptr(), ws.data_ptr(), n, B, hq, nq,
        ctypes.c_float(scale), 1, LIMIT_NS, torch.cuda.current_stream().cuda_stream)
    assert rc == fa.FA_OK
    assert fa.fa_check_device_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_check_device_status() == fa.FA_OK  # the read cleared it
    if prefix:
        o2, lse2 = fa.fa_decode_shared(q, c.k, c.v, c.prefix_pages, prefix, c.tables, c.seq_lens, workspace=ws)
    else:
        o2, lse2 = fa.fa_decode_paged(q, c.k, c.v, c.tables, c.seq_lens, workspace=ws)
    assert fa.fa_check_device_status() == fa.FA_OK
    check_decode(c, q, o2, lse2, scale, heads=[0, hkv - 1], seqs=sorted({0, B // 2, B - 1}))


@pytest.mark.parametrize("bad", [0, -1])
def test_hook_rejects_the_first_tile(bad):
    """Validation comes first: nothing of the call is looked at."""
    lib = fa.load_library()
    assert lib.fa_debug_decode_skip_load(None, None, None, None, 0, None, 1, None, None, None, None, None, 0, 1, 1, 1,
                                         ctypes.c_float(0.1), bad, LIMIT_NS, None) == fa.FA_ERR_INVALID_ARG
