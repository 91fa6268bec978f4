"""What is measured of the paged key/value cache operators.

Three operators of a serving step, in the order in which a step makes them:

* ``append``: the new tokens' keys and values go into a paged cache, the keys
  (and, for the attention that follows, the queries) rotated by their
  positions on the way;
* ``decode``: the new queries of a ragged batch attend to the keys of their
  own sequence in that cache;
* ``shared``: the same for a batch whose sequences continue one common prefix,
  whose pages are read once for all of them.

``run`` computes them in plain torch operations, or, where ``own`` is set, by
the calls that a user of this repository makes.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"

# --------------------------------------------------------------------------- cases


def _case(name, op, **kw):
    c = {
        "name": name, "op": op,
        # heads of the queries and of the cache, head size, rows of a page
        "q_heads": 32, "kv_heads": 8, "d": 128, "page": 64,
        # sequences, new tokens of each (0: a prompt, ragged), tokens in the cache
        "batch": 1, "new": 1, "len_min": 1, "len_max": 1, "len_seed": 1,
        # tokens that all sequences share (shared only)
        "prefix": 0,
        # share of the head that is rotated, and how it is paired (append only)
        "rot": 128, "interleaved": False,
        # order of a page in memory: heads of rows, or rows of heads
        "rows_first": False,
    }
    c.update(kw)
    return c


def listed():
    return [
        # one user's chat: one token of one sequence, where only latency counts
        _case("append_one_token", "append", page=16, len_min=700, len_max=700),
        # a decoding step of a busy server: a token of each of 256 sequences
        _case("append_step_256", "append", batch=256, page=16, len_min=20, len_max=2000, len_seed=2),
        # a scheduler's batch of prompts, ragged, as one packed run of tokens
        _case("append_prompts", "append", batch=12, new=0, len_min=300, len_max=4000, len_seed=3),
        # the same for a smaller model that rotates half of a 64-wide head in
        # neighbouring pairs and keeps the heads of a token together
        _case("append_prompts_d64", "append", batch=7, new=0, q_heads=16, kv_heads=16, d=64, page=32,
              rot=32, interleaved=True, rows_first=True, len_min=99, len_max=5001, len_seed=4),
        # one user's chat: a short cache read once
        _case("decode_one_sequence", "decode", page=16, len_min=701, len_max=701),
        # a busy server's step: sequences of very different lengths
        _case("decode_ragged_48", "decode", batch=48, len_min=100, len_max=9000, len_seed=5),
        # the repository's long decoding workload (8 queries on each of 8 heads
        # against 32768 keys, 8 sequences), from pages
        _case("decode_long_8x32768", "decode", batch=8, q_heads=64, len_min=32768, len_max=32768, page=128),
        # checking four drafted tokens at once; one cache head for each query head, d = 64
        _case("decode_verify_d64", "decode", batch=20, new=4, q_heads=16, kv_heads=16, d=64, page=32,
              len_min=333, len_max=4097, len_seed=6),
        # four answers sampled from one short prompt
        _case("shared_4_answers", "shared", batch=4, prefix=611, len_min=1, len_max=90, len_seed=7, page=16),
        # a system prompt and 32 conversations
        _case("shared_32_chats", "shared", batch=32, prefix=4096, len_min=50, len_max=1500, len_seed=8),
        # many samples of one long problem statement
        _case("shared_128_samples", "shared", batch=128, prefix=16384, len_min=10, len_max=1024, len_seed=9),
        # questions on one long document
        _case("shared_64_questions", "shared", batch=64, q_heads=64, prefix=32768, len_min=100, len_max=700,
              len_seed=10, page=128),
    ]


def lengths(case):
    """Tokens of each sequence's own in the cache after the step (spread over their logarithm)."""
    r = random.Random(case["len_seed"])
    lo, hi = math.log(case["len_min"]), math.log(case["len_max"])
    return [max(case["len_min"], min(case["len_max"], round(math.exp(r.uniform(lo, hi)))))
            for _ in range(case["batch"])]


def new_tokens(case):
    """New tokens of each sequence: `new` of them, or (a prompt) all but a few cached ones."""
    lens = lengths(case)
    if case["new"]:
        return [min(case["new"], n) for n in lens]
    r = random.Random(case["len_seed"] + 1000)
    return [n - r.randint(0, n // 4) for n in lens]


def work(case):
    d, hq, hkv, b = case["d"], case["q_heads"], case["kv_heads"], case["batch"]
    lens = lengths(case)
    if case["op"] == "append":
        t = sum(new_tokens(case))
        # q, k, v in and out, a row of cosines and of sines for each token
        return {"bytes": t * ((hq + 2 * hkv) * d * 4 + 4 * case["rot"]), "flops": 3.0 * t * (hq + hkv) * case["rot"]}
    keys = sum(lens) + case["prefix"]
    rows = b * hq * case["new"]
    n = case["new"]
    pairs = hq * n * (sum(lens) + b * case["prefix"]) - hq * b * n * (n - 1) // 2
    return {"bytes": keys * hkv * d * 4 + rows * (4 * d + 4), "flops": 4.0 * pairs * d}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    caps = {}
    for c in listed():
        w = work(c)
        for k in w:
            caps[c["op"], k] = max(caps.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["append", "decode", "shared"])
        d = rng.choice([64, 128, 128])
        kv = rng.choice([1, 2, 4, 8, 8, 16, 32])
        group = rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
        c = _case("", op, d=d, kv_heads=kv, q_heads=kv * group, page=rng.choice([8, 16, 16, 32, 48, 64, 64, 128, 256]),
                  rows_first=rng.random() < 0.4, len_seed=rng.randrange(1 << 20))
        c["len_max"] = _log_int(rng, 20, 40000)
        c["len_min"] = _log_int(rng, 1, c["len_max"])
        c["batch"] = _log_int(rng, 1, 300)
        if op == "append":
            c["new"] = rng.choice([0, 0, 1, 1, 3])
            c["rot"] = rng.choice([d, d, d // 2, 16, 0])
            c["interleaved"] = rng.random() < 0.4
        else:
            c["new"] = rng.choice([1, 1, 1, 2, 3, 5])
            c["len_min"] = max(c["len_min"], c["new"])
            if group * c["new"] > 64:
                continue
        if op == "shared":
            c["prefix"] = _log_int(rng, 64, 40000)
            c["len_max"] = max(c["len_min"], min(c["len_max"], _log_int(rng, 20, 5000)))
        c["len_max"] = max(c["len_min"], c["len_max"])
        w = work(c)
        plain = c["batch"] * c["len_max"] * kv * d  # elements of the plain form's padded copies
        if all(w[k] <= caps[op, k] for k in w) and plain <= 1 << 29:
            del c["name"]
            return c


# --------------------------------------------------------------------------- inputs


def _pool(case, pages, g):
    """A pool of pages, seen as [pages, heads, rows, d] whatever its order in memory."""
    hkv, rows, d = case["kv_heads"], case["page"], case["d"]
    if case["rows_first"]:
        t = torch.empty((pages, rows, hkv, d), dtype=torch.bfloat16, device=DEVICE).normal_(generator=g)
        return t.permute(0, 2, 1, 3)
    return torch.empty((pages, hkv, rows, d), dtype=torch.bfloat16, device=DEVICE).normal_(generator=g)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    lens, page, b = lengths(case), case["page"], case["batch"]
    need = [-(-n // page) for n in lens]
    prefix_pages = -(-case["prefix"] // page)
    width = max(need)
    total = sum(need) + prefix_pages
    pages = total + 3
    s = {"case": case}
    s["k_pages"] = _pool(case, pages, g)
    s["v_pages"] = _pool(case, pages, g)
    # a pool that has been in use: a sequence's pages lie anywhere in it
    perm = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    idx = torch.zeros((b, width), dtype=torch.int64)
    at = prefix_pages
    for i, n in enumerate(need):
        idx[i, :n] = torch.arange(at, at + n)
        at += n
    s["block_tables"] = perm[idx.to(DEVICE)].contiguous()
    s["prefix_pages"] = perm[:prefix_pages].contiguous()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    if case["op"] == "append":
        new = new_tokens(case)
        cu = torch.zeros(b + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(new), 0).to(torch.int32)
        s["cu_seqlens"] = cu.to(DEVICE)
        t, hq, hkv, d, rot = int(cu[-1]), case["q_heads"], case["kv_heads"], case["d"], case["rot"]
        # the projection's output: q, k and v of a token side by side
        qkv = torch.empty((t, hq + 2 * hkv, d), dtype=torch.bfloat16, device=DEVICE).normal_(generator=g)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["cos"] = s["sin"] = None
        if rot:
            f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
            a = torch.arange(max(lens), dtype=torch.float64, device=DEVICE)[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
    else:
        shape = (b, case["q_heads"], case["new"], case["d"])
        s["q"] = torch.empty(shape, dtype=torch.bfloat16, device=DEVICE).normal_(generator=g)
        s["scale"] = 1.0 / math.sqrt(case["d"])
    return s


# --------------------------------------------------------------------------- plain form


def _token_slots(s):
    """Sequence, cache position, page and row of each new token."""
    cu, lens = s["cu_seqlens"].long(), s["seq_lens"].long()
    t = torch.arange(s["k"].shape[0], device=DEVICE)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = lens[seq] - (cu[seq + 1] - t)
    page = s["k_pages"].shape[2]
    return pos, s["block_tables"].long()[seq, pos // page], pos % page


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[1]
    x = x.float()
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * n, a * n + b * c), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s):
    pos, page, row = _token_slots(s)
    q, k = s["q"], s["k"]
    if s["cos"] is not None:
        cos, sin = s["cos"][pos], s["sin"][pos]
        q = _rotate(q, cos, sin, s["case"]["interleaved"]).to(torch.bfloat16)
        k = _rotate(k, cos, sin, s["case"]["interleaved"]).to(torch.bfloat16)
    else:
        q = q.clone()
    s["k_pages"][page, :, row] = k
    s["v_pages"][page, :, row] = s["v"]
    return q, s["k_pages"], s["v_pages"]


def _rows_of(pages, ids):
    """The rows of the pages `ids` [..., n] in order: [..., heads, n * page, d]."""
    x = pages[ids.long()]  # [..., n, heads, page, d]
    x = x.transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _plain_decode(s):
    q = s["q"].float()
    b, hq, n, d = q.shape
    hkv, page = s["k_pages"].shape[1:3]
    g = hq // hkv
    lens = s["seq_lens"].long()
    k = _rows_of(s["k_pages"], s["block_tables"]).float()  # [b, hkv, m, d]
    m = k.shape[2]
    j = torch.arange(m, device=DEVICE)
    q4 = q.reshape(b, hkv, g * n, d)
    x = torch.matmul(q4, k.transpose(2, 3)).reshape(b, hkv, g, n, m) * s["scale"]
    # query i of the n new ones sees its own key and those before it
    limit = lens[:, None] - n + 1 + torch.arange(n, device=DEVICE)
    x = x.masked_fill(j >= limit[:, None, None, :, None], -math.inf).reshape(b, hkv, g * n, m)
    del k
    p_len = s["case"]["prefix"]
    if p_len:
        kp = _rows_of(s["k_pages"], s["prefix_pages"])[:, :p_len].float()  # [hkv, p, d]
        qh = q4.transpose(0, 1).reshape(hkv, b * g * n, d)
        xp = torch.matmul(qh, kp.transpose(1, 2)).reshape(hkv, b, g * n, p_len) * s["scale"]
        x = torch.cat((xp.transpose(0, 1), x), -1)
        del kp, xp
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = _rows_of(s["v_pages"], s["block_tables"]).float()
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(x[..., p_len:], v)
    del v
    if p_len:
        vp = _rows_of(s["v_pages"], s["prefix_pages"])[:, :p_len].float()
        xp = x[..., :p_len].transpose(0, 1).reshape(hkv, b * g * n, p_len)
        o += torch.matmul(xp, vp).reshape(hkv, b, g * n, d).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.log(total) + top
    return o.reshape(b, hq, n, d).to(torch.bfloat16), lse.reshape(b, hq, n)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import exact_attention_30_gb300 as fa

        if op == "append":
            q = fa.fa_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_tables"], s["seq_lens"],
                                s["cu_seqlens"], q=s["q"], cos=s["cos"], sin=s["sin"],
                                interleaved=s["case"]["interleaved"])
            return q, s["k_pages"], s["v_pages"]
        if op == "decode":
            return fa.fa_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["block_tables"], s["seq_lens"],
                                      s["scale"])
        return fa.fa_decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_pages"], s["case"]["prefix"],
                                   s["block_tables"], s["seq_lens"], s["scale"])
    return _plain_append(s) if op == "append" else _plain_decode(s)


# --------------------------------------------------------------------------- definition


def exact(case, seed):
    """The operators' definitions in 64 bits, token by token or sequence by sequence."""
    s = prepare(case, seed)
    page = case["page"]
    tables = s["block_tables"].tolist()
    lens = lengths(case)
    if case["op"] == "append":
        out_q = s["q"].double()
        out_k, out_v = s["k_pages"].double(), s["v_pages"].double()
        half = case["rot"] // 2
        first = [2 * i if case["interleaved"] else i for i in range(half)]
        second = [2 * i + 1 if case["interleaved"] else i + half for i in range(half)]
        start = 0
        for b, n in enumerate(new_tokens(case)):
            at = list(range(lens[b] - n, lens[b]))
            k, v = s["k"][start:start + n].double(), s["v"][start:start + n].double()
            if half:
                c, z = s["cos"][at].double()[:, None], s["sin"][at].double()[:, None]
                for x in (k, out_q[start:start + n]):
                    u, w = x[..., first], x[..., second]
                    x[..., first], x[..., second] = u * c - w * z, u * z + w * c
            ids = torch.tensor([tables[b][p // page] for p in at], device=DEVICE)
            rows = torch.tensor([p % page for p in at], device=DEVICE)
            out_k[ids, :, rows], out_v[ids, :, rows] = k, v
            start += n
        return out_q, out_k, out_v
    q = s["q"].double()
    b_n, hq, n, d = q.shape
    hkv = case["kv_heads"]
    p_len = case["prefix"]
    if p_len:
        ids = s["prefix_pages"].long()
        kp = torch.cat([s["k_pages"][i] for i in ids], 1)[:, :p_len].double()
        vp = torch.cat([s["v_pages"][i] for i in ids], 1)[:, :p_len].double()
    o = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device=DEVICE)
    for b in range(b_n):
        ids = torch.tensor(tables[b][:-(-lens[b] // page)], device=DEVICE)
        k = torch.cat(list(s["k_pages"][ids]), 1)[:, :lens[b]].double()
        v = torch.cat(list(s["v_pages"][ids]), 1)[:, :lens[b]].double()
        if p_len:
            k, v = torch.cat((kp, k), 1), torch.cat((vp, v), 1)
        qb = q[b].reshape(hkv, hq // hkv, n, d)
        for i in range(n):
            seen = p_len + max(0, lens[b] - n + 1 + i)
            if not seen:
                lse[b, :, i] = -math.inf
                continue
            x = torch.einsum("hgd,hkd->hgk", qb[:, :, i], k[:, :seen]) * s["scale"]
            lse[b, :, i] = torch.logsumexp(x, -1).reshape(hq)
            o[b, :, i] = torch.einsum("hgk,hkd->hgd", torch.softmax(x, -1), v[:, :seen]).reshape(hq, d)
    return o, lse
