"""What is measured of the prompt operators and of eviction from the paged cache.

Five operators, in the order in which a program that trains or serves with
grouped heads makes them:

* ``prompt``: causal attention of packed prompts of different lengths, several
  query heads on one key/value head; the keys packed as the queries are, or
  (a chat's next turn) in the pages of a cache that already holds more;
* ``grad``: its backward pass, the gradients of a shared head summed;
* ``weights``: the attention weight that each key of a prompt got, summed over
  the queries (all of them, or a window of the last ones) and the query heads;
* ``step``: the same for the new tokens of a decoding step over a paged cache;
* ``evict``: of each sequence and key/value head, the keys with the largest
  weights and the newest ones stay, and move together into fewer pages.

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
        # heads of the queries and of the keys, head size
        "q_heads": 32, "kv_heads": 8, "d": 128,
        # sequences, new tokens of each, tokens before them in the cache
        "batch": 1, "new_min": 1, "new_max": 1, "past_min": 0, "past_max": 0, "len_seed": 1,
        # rows of a page (0: packed keys), and whether a page holds rows of heads
        "page": 0, "rows_first": False,
        # queries that count (weights only; 0: all)
        "window": 0,
        # keys that stay, and how many of them are the newest ones (evict only)
        "budget": 0, "recent": 0,
    }
    c.update(kw)
    return c


def listed():
    return [
        # one user's short question, where only latency counts
        _case("prompt_one_question", "prompt", new_min=37, new_max=37),
        # a scheduler's batch of prompts of very different lengths
        _case("prompt_ragged_16", "prompt", batch=16, new_min=100, new_max=8000, len_seed=2),
        # one long document, heads as in the repository's workload of 16384 rows, four to a key/value head
        _case("prompt_document_32768", "prompt", new_min=32768, new_max=32768),
        # the next turn of some chats of a smaller model, whose earlier turns are in the cache
        _case("prompt_next_turns_d64", "prompt", batch=6, q_heads=16, kv_heads=4, d=64, new_min=20, new_max=700,
              past_min=1000, past_max=20000, len_seed=5, page=32, rows_first=True),
        # fine-tuning a smaller model, seven query heads to a 64-wide key/value head, on a few short examples
        _case("grad_short_examples_d64", "grad", batch=5, q_heads=14, kv_heads=2, d=64, new_min=9, new_max=300, len_seed=2),
        # a training step's packed batch
        _case("grad_packed_8", "grad", batch=8, new_min=500, new_max=4096, len_seed=5),
        # how much attention each token of a batch of prompts got
        _case("weights_prompts_8", "weights", batch=8, new_min=300, new_max=8000, len_seed=2),
        # the same by the last 64 tokens of long prompts
        _case("weights_window_64", "weights", batch=6, new_min=5000, new_max=20000, window=64, len_seed=8),
        # checking four drafted tokens of one chat
        _case("step_one_chat_d64", "step", q_heads=16, kv_heads=4, d=64, new_min=4, new_max=4, past_min=700, past_max=700,
              page=16),
        # a busy server's step: one token of each sequence
        _case("step_ragged_48", "step", batch=48, past_min=100, past_max=9000, len_seed=9, page=64),
        # every 64 steps, 64 chats are cut back to 1024 keys
        _case("evict_64_chats", "evict", batch=64, past_min=1088, past_max=1088, budget=1024, recent=128, page=64),
        # after long prompts, ragged
        _case("evict_after_prompts", "evict", batch=8, past_min=3000, past_max=32768, budget=2048, recent=64, page=16,
              len_seed=10),
    ]


def _spread(r, lo, hi, n):
    """n whole numbers from lo to hi, spread over their logarithm (from one less than lo = 0 on)."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [max(lo, min(hi, round(math.exp(r.uniform(a, b)) - 1))) for _ in range(n)]


def lengths(case):
    """New tokens of each sequence, and its keys after the step."""
    r = random.Random(case["len_seed"])
    new = _spread(r, case["new_min"], case["new_max"], case["batch"])
    past = _spread(r, case["past_min"], case["past_max"], case["batch"])
    if case["op"] == "evict":
        return new, past
    return new, [n + p for n, p in zip(new, past)]


def _pairs(case):
    """(query token, key) pairs that attend."""
    new, keys = lengths(case)
    if case["window"]:
        new = [min(n, case["window"]) for n in new]
    return sum(n * m - n * (n - 1) // 2 for n, m in zip(new, keys))


def work(case):
    d, hq, hkv = case["d"], case["q_heads"], case["kv_heads"]
    new, keys = lengths(case)
    rows, t_k = hq * sum(new), hkv * sum(keys)
    op = case["op"]
    if op == "prompt":
        return {"bytes": rows * (4 * d + 4) + t_k * 4 * d, "flops": 4.0 * d * hq * _pairs(case)}
    if op == "grad":
        return {"bytes": rows * (8 * d + 4) + t_k * 8 * d, "flops": 10.0 * d * hq * _pairs(case)}
    if op in ("weights", "step"):
        if case["window"]:
            rows = hq * sum(min(n, case["window"]) for n in new)
        return {"bytes": rows * (2 * d + 4) + t_k * (2 * d + 4), "flops": 2.0 * d * hq * _pairs(case)}
    kept = hkv * sum(min(m, case["budget"]) for m in keys)
    # the weights, the kept keys and values in and out, their weights and indices
    return {"bytes": 4 * t_k + kept * (8 * d + 8), "flops": 4.0 * t_k}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    caps = {}
    for c in listed():
        w = work(c)
        for k in w:
            caps[c["op"], k] = max(caps.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["prompt", "prompt", "grad", "grad", "weights", "step", "evict"])
        kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16])
        c = _case("", op, d=rng.choice([64, 128, 128]), kv_heads=kv, q_heads=kv * group, len_seed=rng.randrange(1 << 20),
                  batch=_log_int(rng, 1, 100))
        if op in ("prompt", "grad", "weights"):
            c["new_max"] = _log_int(rng, 1, 20000)
            c["new_min"] = _log_int(rng, 1, c["new_max"])
            if op != "weights" and rng.random() < 0.4:
                c["past_max"] = _log_int(rng, 1, 20000)
                c["past_min"] = rng.choice([0, _log_int(rng, 1, c["past_max"])])
        if op == "weights":
            c["window"] = rng.choice([0, 0, 1, 16, 32, 64, 100])
        if op == "step":
            c["new_min"] = c["new_max"] = rng.choice([1, 1, 1, 2, 4])
            c["past_max"] = _log_int(rng, 20, 40000)
            c["past_min"] = rng.choice([0, _log_int(rng, 1, c["past_max"])])
            if group * c["new_max"] > 64:
                continue
        if op == "evict":
            c["past_max"] = _log_int(rng, 20, 40000)
            c["past_min"] = _log_int(rng, 1, c["past_max"])
            c["budget"] = _log_int(rng, 1, c["past_max"])
            c["recent"] = rng.choice([0, 1, c["budget"] // 4, c["budget"]])
        if op in ("step", "evict") or (op == "prompt" and rng.random() < 0.5):
            c["page"] = rng.choice([8, 16, 16, 32, 48, 64, 64, 128, 256])
            c["rows_first"] = rng.random() < 0.4
        w = work(c)
        new, keys = lengths(c)
        if op == "grad" and max(keys) < 2:
            continue  # a single key has all the weight: these gradients are zero
        if all(w[k] <= caps[op, k] for k in w) and len(keys) * max(keys) * kv * c["d"] <= 1 << 29:
            del c["name"]
            return c


# --------------------------------------------------------------------------- inputs


def _normal(shape, g):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEVICE).normal_(generator=g)


def _offsets(lens):
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0).to(torch.int32)
    return cu.to(DEVICE)


def _pool(case, pages, g):
    """A pool of pages, seen as [pages, heads, rows, d] whatever its order in memory."""
    hkv, rows, d = case["kv_heads"], case["page"], case["d"]
    if case["rows_first"]:
        return _normal((pages, rows, hkv, d), g).permute(0, 2, 1, 3)
    return _normal((pages, hkv, rows, d), g)


def _tables(first, need, perm):
    """A table of pages: sequence i owns need[i] pages of the pool, which lie anywhere in it."""
    idx = torch.zeros((len(need), max(max(need), 1)), dtype=torch.int64)
    for i, n in enumerate(need):
        idx[i, :n] = torch.arange(first, first + n)
        first += n
    return perm[idx.to(DEVICE)].contiguous(), first


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    new, keys = lengths(case)
    b, hq, hkv, d, page = case["batch"], case["q_heads"], case["kv_heads"], case["d"], case["page"]
    op = case["op"]
    s = {"case": case, "new": new, "keys": keys, "scale": 1.0 / math.sqrt(d)}
    if page:
        need = [-(-m // page) for m in keys]
        after = [-(-min(m, case["budget"]) // page) for m in keys] if op == "evict" else []
        pages = sum(need) + sum(after) + 3
        s["k_pages"], s["v_pages"] = _pool(case, pages, g), _pool(case, pages, g)
        # a pool that has been in use: a sequence's pages lie anywhere in it
        perm = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
        s["block_tables"], used = _tables(0, need, perm)
        s["seq_lens"] = torch.tensor(keys, dtype=torch.int32, device=DEVICE)
        if op == "evict":
            s["new_tables"], _ = _tables(used, after, perm)
    if op == "evict":
        shape = (b, hkv, max(keys))
        # few keys hold most of the weight, and many got none that counts
        w = torch.empty(shape, dtype=torch.float32, device=DEVICE).normal_(generator=g).mul_(2).exp_()
        s["weights"] = torch.where(w < 0.2, 0.0, w)
        s["new_weights"] = torch.zeros((b, hkv, case["budget"]), dtype=torch.float32, device=DEVICE)
        return s
    if op == "step":
        s["q"] = _normal((b, hq, case["new_max"], d), g)
        s["weights"] = torch.zeros((b, hkv, max(keys)), dtype=torch.float32, device=DEVICE)
        s["lse"] = _plain_step_lse(s)
        return s
    t, t_k = sum(new), sum(keys)
    s["cu_q"] = _offsets(new)
    s["cu_k"] = _offsets(keys)
    if t == t_k and not page:  # the projection's output: q, k and v of a token side by side
        qkv = _normal((t, hq + 2 * hkv, d), g)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"] = _normal((t, hq, d), g)
        if not page:
            s["k"], s["v"] = _normal((t_k, hkv, d), g), _normal((t_k, hkv, d), g)
    if op == "grad":
        s["do"] = _normal((t, hq, d), g)
        s["o"], s["lse"] = _plain_prompt(s)
    if op == "weights":
        s["weights"] = torch.zeros((b, hkv, max(keys)), dtype=torch.float32, device=DEVICE)
        s["lse"] = _plain_prompt_lse(s)
    return s


# --------------------------------------------------------------------------- plain form

_MOST = 1 << 29  # scores at a time


def _rows_of(pages, ids):
    """The rows of the pages `ids` [..., n] in order: [..., heads, n * page, d]."""
    x = pages[ids.long()].transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _sequences(s):
    """Of each sequence: its first token, tokens and keys, and the keys and values in 32 bits, [heads, keys, d]."""
    at = at_k = 0
    for i, (n, m) in enumerate(zip(s["new"], s["keys"])):
        if n and m:
            if "k" in s:
                k, v = (s[x][at_k:at_k + m].transpose(0, 1).float() for x in ("k", "v"))
            else:
                k, v = (_rows_of(s[x], s["block_tables"][i])[:, :m].float() for x in ("k_pages", "v_pages"))
            yield i, at, n, m, k, v
        at += n
        at_k += m


def _parts(first, n, m, hq):
    """Runs of the queries from `first` on of a sequence whose scores can be held at once: first, end, keys that they see."""
    step = max(1, _MOST // (hq * m))
    for a in range(first, n, step):
        e = min(n, a + step)
        yield a, e, m - n + e


def _scores(s, q, k, a, e, n, m, seen):
    """Scaled scores of queries a .. e - 1 of a sequence, [heads, group, queries, keys], -inf where a key is later."""
    hkv, hq, d = k.shape[0], q.shape[1], q.shape[2]
    q4 = q.float().reshape(e - a, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    x = torch.matmul(q4, k[:, :seen].transpose(1, 2)).mul_(s["scale"]).reshape(hkv, hq // hkv, e - a, seen)
    later = torch.arange(seen, device=DEVICE) > torch.arange(a + m - n, e + m - n, device=DEVICE)[:, None]
    return x.masked_fill_(later, -math.inf)


def _tokens_first(x):
    """[heads, group, queries, ...] as [queries, heads * group, ...]."""
    return x.flatten(0, 1).transpose(0, 1)


def _plain_prompt(s):
    q = s["q"]
    t, hq, d = q.shape
    o = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEVICE)
    lse = torch.empty((hq, t), dtype=torch.float32, device=DEVICE)
    for _, at, n, m, k, v in _sequences(s):
        for a, e, seen in _parts(0, n, m, hq):
            x = _scores(s, q[at + a:at + e], k, a, e, n, m, seen)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            y = torch.matmul(x.flatten(1, 2), v[:, :seen]).reshape(*x.shape[:3], d) / total
            o[at + a:at + e] = _tokens_first(y)
            lse[:, at + a:at + e] = (total.log() + top).flatten(0, 1).squeeze(-1)
    return o, lse


def _plain_prompt_lse(s):
    lse = torch.empty((s["q"].shape[1], s["q"].shape[0]), dtype=torch.float32, device=DEVICE)
    for _, at, n, m, k, _ in _sequences(s):
        for a, e, seen in _parts(0, n, m, lse.shape[0]):
            x = _scores(s, s["q"][at + a:at + e], k, a, e, n, m, seen)
            lse[:, at + a:at + e] = torch.logsumexp(x, -1).flatten(0, 1)
    return lse


def _heads_first(x, hkv):
    """[queries, heads * group, ...] in 32 bits as [heads, group * queries, ...]."""
    n, hq = x.shape[:2]
    return x.float().transpose(0, 1).reshape(hkv, hq // hkv * n, *x.shape[2:])


def _plain_grad(s):
    q, o, do, lse = s["q"], s["o"], s["do"], s["lse"]
    hkv, scale = s["k"].shape[1], s["scale"]
    dq = torch.empty(q.shape, dtype=torch.bfloat16, device=DEVICE)
    dk = torch.empty(s["k"].shape, dtype=torch.bfloat16, device=DEVICE)
    dv = torch.empty_like(dk)
    at_k = 0
    for _, at, n, m, k, v in _sequences(s):
        gk, gv = torch.zeros_like(k), torch.zeros_like(v)
        for a, e, seen in _parts(0, n, m, q.shape[1]):
            rows = slice(at + a, at + e)
            p = _scores(s, q[rows], k, a, e, n, m, seen)
            p = p.sub_(lse[:, rows].reshape(hkv, -1, e - a, 1)).exp_().flatten(1, 2)
            qh, gh = _heads_first(q[rows], hkv), _heads_first(do[rows], hkv)
            delta = (gh * _heads_first(o[rows], hkv)).sum(-1, keepdim=True)
            gv[:, :seen] += torch.matmul(p.transpose(1, 2), gh)
            ds = torch.matmul(gh, v[:, :seen].transpose(1, 2)).sub_(delta).mul_(p).mul_(scale)
            del p
            gk[:, :seen] += torch.matmul(ds.transpose(1, 2), qh)
            gq = torch.matmul(ds, k[:, :seen]).reshape(hkv, -1, e - a, q.shape[2])
            dq[rows] = _tokens_first(gq)
            del ds
        dk[at_k:at_k + m], dv[at_k:at_k + m] = gk.transpose(0, 1), gv.transpose(0, 1)
        at_k += m
    return dq, dk, dv


def _plain_weights(s):
    w, lse = s["weights"], s["lse"]
    hkv, window = w.shape[1], s["case"]["window"]
    for i, at, n, m, k, _ in _sequences(s):
        w[i, :, :m] = 0
        for a, e, seen in _parts(max(0, n - window) if window else 0, n, m, lse.shape[0]):
            x = _scores(s, s["q"][at + a:at + e], k, a, e, n, m, seen)
            x = x.sub_(lse[:, at + a:at + e].reshape(hkv, -1, e - a, 1)).exp_()
            w[i, :, :seen] += x.sum((1, 2))
    return w


def _step_scores(s):
    """Scaled scores of a step, [batch, heads, group, new, keys], -inf for keys that a token does not see."""
    q, lens = s["q"].float(), s["seq_lens"].long()
    b, hq, n, d = q.shape
    hkv = s["k_pages"].shape[1]
    m = s["weights"].shape[2]
    k = _rows_of(s["k_pages"], s["block_tables"])[:, :, :m].float()
    x = torch.matmul(q.reshape(b, hkv, -1, d), k.transpose(2, 3)).mul_(s["scale"]).reshape(b, hkv, hq // hkv, n, m)
    limit = lens[:, None] - n + 1 + torch.arange(n, device=DEVICE)
    return x.masked_fill_(torch.arange(m, device=DEVICE) >= limit[:, None, None, :, None], -math.inf)


def _plain_step_lse(s):
    return torch.logsumexp(_step_scores(s), -1).flatten(1, 2)


def _plain_step(s):
    x = _step_scores(s)
    x = x.sub_(s["lse"].reshape(*x.shape[:4], 1)).exp_().sum((2, 3))
    inside = torch.arange(x.shape[2], device=DEVICE) < s["seq_lens"].long()[:, None, None]
    s["weights"].copy_(torch.where(inside, x, s["weights"]))
    return s["weights"]


def _plain_evict(s):
    w, lens = s["weights"], s["seq_lens"].long()
    b, hkv, m = w.shape
    budget, recent, page = s["case"]["budget"], s["case"]["recent"], s["case"]["page"]
    j = torch.arange(m, device=DEVICE)
    count = lens.clamp(max=budget)[:, None, None]
    key = torch.where(j >= (lens - recent)[:, None, None], math.inf, w)
    key = torch.where(j < lens[:, None, None], key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    rank = torch.arange(order.shape[-1], device=DEVICE)
    order = torch.sort(torch.where(rank < count, order, m), -1).values
    kept = torch.full((b, hkv, budget), -1, dtype=torch.int32, device=DEVICE)
    kept[..., :order.shape[-1]] = torch.where(rank < count, order, -1)
    # rows past a sequence's last one are taken for its last one
    rank = torch.minimum(rank, count - 1).expand(b, hkv, -1)
    src = torch.gather(order, -1, rank)
    seq, head = torch.arange(b, device=DEVICE)[:, None, None], torch.arange(hkv, device=DEVICE)[:, None]
    from_page, to_page = s["block_tables"].long()[seq, src // page], s["new_tables"].long()[seq, rank // page]
    for x in (s["k_pages"], s["v_pages"]):
        x[to_page, head, rank % page] = x[from_page, head, src % page]
    s["new_weights"][seq, head, rank] = w[seq, head, src]
    return count.flatten().to(torch.int32), kept, s["new_weights"], s["k_pages"], s["v_pages"]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import exact_attention_30_gb300 as fa

        n, m = max(s["new"]), max(s["keys"])
        if op == "prompt" and "k" in s:
            return fa.fa_prompt_fwd(s["q"], s["k"], s["v"], s["cu_q"], n, s["cu_k"], m, scale=s["scale"])
        if op == "prompt":
            return fa.fa_prompt_paged(s["q"], s["k_pages"], s["v_pages"], s["block_tables"], s["seq_lens"], s["cu_q"], n,
                                      scale=s["scale"])
        if op == "grad":
            return fa.fa_prompt_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["cu_q"], n, s["cu_k"], m,
                                    scale=s["scale"])
        if op == "weights":
            return fa.fa_prompt_key_weights(s["q"], s["k"], s["lse"], s["weights"], s["cu_q"], n, s["cu_k"], m,
                                            window=s["case"]["window"], scale=s["scale"])
        if op == "step":
            return fa.fa_decode_key_weights(s["q"], s["k_pages"], s["block_tables"], s["seq_lens"], s["lse"],
                                            s["weights"], accumulate=False, scale=s["scale"])
        lens, kept = fa.fa_kv_evict(s["k_pages"], s["v_pages"], s["block_tables"], s["seq_lens"], s["weights"],
                                    s["case"]["budget"], s["case"]["recent"], new_tables=s["new_tables"],
                                    new_weights=s["new_weights"])
        return lens, kept, s["new_weights"], s["k_pages"], s["v_pages"]
    if op == "prompt":
        return _plain_prompt(s)
    if op == "grad":
        return _plain_grad(s)
    if op == "weights":
        return _plain_weights(s)
    return _plain_step(s) if op == "step" else _plain_evict(s)


# --------------------------------------------------------------------------- definition


def exact(case, seed):
    """The operators' definitions in 64 bits, a sequence and a key/value head (or a few of its queries) at a time."""
    # products in 64 bits: about one TFLOP in a second
    if {"prompt": 2, "grad": 5, "weights": 2, "step": 1, "evict": 0}[case["op"]] * 2.0 * case["d"] * case["q_heads"] * \
            _pairs(case) > 1e13:
        return None
    s = prepare(case, seed)
    new, keys = lengths(case)
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["d"], case["page"]
    group = hq // hkv
    f64 = {"dtype": torch.float64, "device": DEVICE}
    if case["op"] == "evict":
        kept = torch.full((case["batch"], hkv, case["budget"]), -1, dtype=torch.int32)
        w = s["weights"].cpu().tolist()
        out_k, out_v, out_w = s["k_pages"].double(), s["v_pages"].double(), s["new_weights"].double()
        for i, m in enumerate(keys):
            c = min(m, case["budget"])
            old = m - min(case["recent"], m)
            at = torch.arange(c, device=DEVICE)
            for h in range(hkv):
                best = sorted(range(old), key=lambda j: (-w[i][h][j], j))[:max(0, c - (m - old))]
                stay = torch.tensor((sorted(best) + list(range(old, m)))[-c:], device=DEVICE)
                kept[i, h, :c] = stay.to(torch.int32).cpu()
                for x, y in ((s["k_pages"], out_k), (s["v_pages"], out_v)):
                    y[s["new_tables"][i][at // page].long(), h, at % page] = \
                        x[s["block_tables"][i][stay // page].long(), h, stay % page].double()
                out_w[i, h, :c] = s["weights"][i, h][stay].double()
        lens = torch.tensor([min(m, case["budget"]) for m in keys], dtype=torch.int32)
        return lens, kept, out_w, out_k, out_v
    starts_q = [sum(new[:i]) for i in range(len(new))]
    starts_k = [sum(keys[:i]) for i in range(len(keys))]
    t = sum(new)
    o, lse = torch.zeros((t, hq, d), **f64), torch.zeros((hq, t), **f64)
    dq = torch.zeros((t, hq, d), **f64)
    dk, dv = torch.zeros((sum(keys), hkv, d), **f64), torch.zeros((sum(keys), hkv, d), **f64)
    weights = s["weights"].double() if "weights" in s else None
    for i, (n, m) in enumerate(zip(new, keys)):
        for h in range(hkv if n else 0):
            if page:
                ids = s["block_tables"][i][:-(-m // page)].long()
                k = torch.cat(list(s["k_pages"][ids, h]))[:m].double()
                v = torch.cat(list(s["v_pages"][ids, h]))[:m].double()
            else:
                k = s["k"][starts_k[i]:starts_k[i] + m, h].double()
                v = s["v"][starts_k[i]:starts_k[i] + m, h].double()
            if weights is not None:
                weights[i, h, :m] = 0
            for g in range(h * group, (h + 1) * group):
                step = max(1, (1 << 27) // m)
                for a in range(0, n, step):
                    e = min(n, a + step)
                    r = slice(starts_q[i] + a, starts_q[i] + e)
                    q = s["q"][i, g, a:e] if case["op"] == "step" else s["q"][r, g]
                    x = (q.double() @ k.T) * s["scale"]
                    token = torch.arange(a, e, device=DEVICE)[:, None]
                    x = torch.where(torch.arange(m, device=DEVICE) <= token + (m - n), x, -math.inf)
                    if weights is not None:
                        z = s["lse"][i, g, a:e] if case["op"] == "step" else s["lse"][g, r]
                        p = torch.exp(x - z.double()[:, None])
                        if case["window"]:
                            p = torch.where(token >= n - case["window"], p, 0.0)
                        weights[i, h, :m] += p.sum(0)
                        continue
                    lse[g, r] = torch.logsumexp(x, -1)
                    p = torch.softmax(x, -1)
                    o[r, g] = p @ v
                    if case["op"] == "grad":
                        y = s["do"][r, g].double()
                        dp = y @ v.T
                        ds = p * (dp - (dp * p).sum(-1, keepdim=True)) * s["scale"]
                        rows = slice(starts_k[i], starts_k[i] + m)
                        dv[rows, h] += p.T @ y
                        dk[rows, h] += ds.T @ q.double()
                        dq[r, g] = ds @ k
    if weights is not None:
        return weights
    return (dq, dk, dv) if case["op"] == "grad" else (o, lse)
