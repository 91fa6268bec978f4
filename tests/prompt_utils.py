"""Packed prompts with grouped heads, and the plain fp64 definitions the prompt operators are tested against."""
import math

import torch

EPS_BF16 = 2.0 ** -8   # half a step of bf16, relative (rounding to nearest)
EPS_F32 = 2.0 ** -24
TINY = 2.0 ** -126


def bf16_randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def offsets(lens, first=0):
    return torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()


class Prompts:
    """A packed batch: sequence b has n[b] tokens and m[b] keys. `pad`: padding tokens before the
    first sequence and behind the last one, NaN in the inputs. `fused`: q, k and v are slices of one
    projection's output (n = m)."""

    def __init__(self, n, hq, hkv, d, m=None, seed=0, pad=(0, 0), fused=False, big=0):
        self.n, self.m = list(n), list(n) if m is None else list(m)
        self.hq, self.hkv, self.d, self.g = hq, hkv, d, hq // hkv
        self.pad = pad
        t, tk = sum(self.n) + sum(pad), sum(self.m) + sum(pad)
        self.total, self.total_k = t, tk
        if fused:
            qkv = bf16_randn((t, hq + 2 * hkv, d), seed)
            self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            self.q, self.k, self.v = (bf16_randn(s, seed + i) for i, s in
                                      enumerate(((t, hq, d), (tk, hkv, d), (tk, hkv, d))))
        if big:
            self.k[::big] *= 4
        self.do = bf16_randn((t, hq, d), seed + 7)
        a, z = pad
        for x in (self.q, self.k, self.v, self.do):
            x[:a] = math.nan
            x[x.shape[0] - z:] = math.nan
        self.cu_q, self.cu_k = offsets(self.n, a), offsets(self.m, a)
        self.max_q, self.max_k = max(self.n + [1]), max(self.m + [1])

    def seqs(self):
        at, at_k = self.pad[0], self.pad[0]
        for b, (n, m) in enumerate(zip(self.n, self.m)):
            yield b, slice(at, at + n), slice(at_k, at_k + m), n, m
            at += n
            at_k += m

    def head(self, b, rows, keys, h):
        """(q [g, n, d], k, v) in fp64 of K/V head h of a sequence."""
        q = self.q[rows, h * self.g:(h + 1) * self.g].transpose(0, 1).cpu().double()
        return q, self.k[keys, h].cpu().double(), self.v[keys, h].cpu().double()


class Paged(Prompts):
    """Prompts whose keys are in a paged cache."""

    def __init__(self, n, cache, hq, seed=0, pad=(0, 0)):
        self.n, self.m, self.cache = list(n), cache.lens, cache
        self.hq, self.hkv, self.d, self.g, self.pad = hq, cache.hkv, cache.d, hq // cache.hkv, pad
        self.total = sum(n) + sum(pad)
        self.q = bf16_randn((self.total, hq, cache.d), seed)
        self.cu_q = offsets(self.n, pad[0])

    def head(self, b, rows, keys, h):
        q = self.q[rows, h * self.g:(h + 1) * self.g].transpose(0, 1).cpu().double()
        k, v = self.cache.keys_values(b, h)
        return q, torch.from_numpy(k), torch.from_numpy(v)


def seen_mask(n, m):
    """[n, m] True where token i of n sees key j of m."""
    return torch.arange(m) <= torch.arange(n)[:, None] + (m - n)


def attention64(q, k, v, scale):
    """O [.., n, d], LSE [.., n], P [.., n, m] in fp64; a row without keys: 0, -inf, 0."""
    n, m = q.shape[-2], k.shape[-2]
    x = q @ k.transpose(-1, -2) * scale
    x = torch.where(seen_mask(n, m), x, -math.inf)
    if m == 0:
        return torch.zeros_like(q), torch.full(q.shape[:-1], -math.inf, dtype=q.dtype), x
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    s = e.sum(-1, keepdim=True)
    p = torch.where(s > 0, e / s, 0.0)
    return p @ v, (torch.log(s) + top).squeeze(-1), p


def score_error(q, k, scale, d):
    """Bound of a score's error in fp32 and of what the exponential adds: d products summed in any
    order, (d + 8) 2^-24 scale sum |q k|, and 2^-19 relative for exponentials and merges."""
    if k.shape[-2] == 0 or q.shape[-2] == 0:
        return 2.0 ** -19
    return (d + 8) * EPS_F32 * scale * (q.abs() @ k.abs().transpose(-1, -2)).max().item() + 2.0 ** -19


def check_forward(c, o, lse, scale, heads=None, seqs=None):
    """Every row against the definition. O is rounded to bf16 once (half a step of |o|), every weight
    of P V once (at most half a step of sum_j p_j |v_j|), and scores and exponentials add e, which
    enters the numerator and the denominator."""
    for b, rows, keys, n, m in c.seqs():
        if seqs is not None and b not in seqs:
            continue
        for h in range(c.hkv) if heads is None else heads:
            q, k, v = c.head(b, rows, keys, h)
            ref, ref_l, p = attention64(q, k, v, scale)
            e = score_error(q, k, scale, c.d)
            got = o[rows, h * c.g:(h + 1) * c.g].transpose(0, 1).cpu().double()
            got_l = lse[h * c.g:(h + 1) * c.g, rows].cpu().double()
            size = p @ v.abs() if m else torch.zeros_like(ref)
            tol = EPS_BF16 * ref.abs() + (1.01 * EPS_BF16 + 2 * e) * size
            err = (got - ref).abs()
            assert torch.isfinite(got).all(), (b, h)
            assert (err <= tol).all(), (b, h, (err / tol.clamp(min=1e-30)).max())
            none = ref_l == -math.inf
            assert ((got_l == -math.inf) == none).all(), (b, h)
            dl = torch.where(none, 0.0, (got_l - ref_l).abs())
            assert (dl <= e + torch.where(none, 0.0, ref_l.abs()) * 2.0 ** -22 + 2.0 ** -19).all(), (b, h, dl.max())


def backward64(q, k, v, do, scale):
    """dQ [g, n, d], dK, dV [m, d] (summed over g) in fp64, and what their tolerances count: P, dP - D, and
    the sizes sum |dO| |O'| with O' the bound of O's own error per element."""
    o, _, p = attention64(q, k, v, scale)
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), p, p, None
    dp = do @ v.transpose(-1, -2)
    t = torch.where(p > 0, dp - (do * o).sum(-1, keepdim=True), 0.0)
    ds = p * t * scale
    d_err = (do.abs() * (EPS_BF16 * o.abs() + 1.02 * EPS_BF16 * (p @ v.abs()))).sum(-1, keepdim=True)
    return ds @ k, (ds.transpose(-1, -2) @ q).sum(0), (p.transpose(-1, -2) @ do).sum(0), p, t, d_err


def check_backward(c, dq, dk, dv, scale, seqs=None):
    """Every gradient against the formula. P and dS are rounded to bf16 once for their products, each
    gradient once at the end (half a step each); O, rounded like that, enters through D = sum dO O; scores
    and exponentials add e to P (score_error), products of d terms in fp32 (d + 8) 2^-24 of their sizes, and
    sums over queries or keys 2^-18. A P below 2^-126, fp32's least normal number, becomes zero in the
    exponential, which moves it by at most that, and so may a gradient below it."""
    for b, rows, keys, n, m in c.seqs():
        if seqs is not None and b not in seqs:
            continue
        for h in range(c.hkv):
            q, k, v = c.head(b, rows, keys, h)
            hs = slice(h * c.g, (h + 1) * c.g)
            do = c.do[rows, hs].transpose(0, 1).cpu().double()
            rq, rk, rv, p, t, d_err = backward64(q, k, v, do, scale)
            got_q = dq[rows, hs].transpose(0, 1).cpu().double()
            got_k, got_v = dk[keys, h].cpu().double(), dv[keys, h].cpu().double()
            if m == 0 or n == 0:
                assert (got_q == 0).all() and (got_k == 0).all() and (got_v == 0).all(), (b, h)
                continue
            r = 1.01 * EPS_BF16 + 2 * score_error(q, k, scale, c.d) + 2.0 ** -18
            dp_err = (c.d + 8) * EPS_F32 * 2 * (do.abs() @ v.abs().transpose(-1, -2)) + d_err
            t_all = (do @ v.transpose(-1, -2)).abs() + (do.abs() * (p @ v).abs()).sum(-1, keepdim=True)
            ds_err = scale * (p * (t.abs() * r + dp_err * (1 + r)) + TINY * seen_mask(n, m) * (t_all + dp_err))
            size_v = (p.transpose(-1, -2) @ do.abs()).sum(0)
            tiny_v = TINY * (seen_mask(n, m).double().T @ do.abs()).sum(0)
            for name, got, ref, tol in (("dq", got_q, rq, ds_err @ k.abs()),
                                        ("dk", got_k, rk, (ds_err.transpose(-1, -2) @ q.abs()).sum(0)),
                                        ("dv", got_v, rv, r * size_v + tiny_v)):
                tol = tol + EPS_BF16 * 1.01 * ref.abs() + TINY
                err = (got - ref).abs()
                assert torch.isfinite(got).all(), (b, h, name)
                assert (err <= tol).all(), (b, h, name, (err / tol.clamp(min=1e-30)).max(), (err > tol).sum())


def check_weights(c, w, before, lse, scale, window=0, accumulate=True, seqs=None):
    """Every key's weight against the definition, with the fp32 lse that the call had. Each weight of a query is off
    by e (score_error, twice: it is an exponent) and 2^-17 relative (the exponential, the rounding of -LSE * log2(e)
    and of its sum with a score, and the sums); what was there is added in fp32."""
    for b, rows, keys, n, m in c.seqs():
        if seqs is not None and b not in seqs:
            continue
        for h in range(c.hkv):
            got, old = w[b, h].cpu().double(), before[b, h].cpu().double()
            if n == 0:
                assert torch.equal(got, old), (b, h)
                continue
            q, k, _ = c.head(b, rows, keys, h)
            z = lse[h * c.g:(h + 1) * c.g, rows].cpu().double()
            x = torch.where(seen_mask(n, m), q @ k.transpose(-1, -2) * scale, -math.inf)
            p = torch.where(z[..., None] == -math.inf, 0.0, torch.exp(x - z[..., None]))
            if window:
                p[:, :max(0, n - window)] = 0
            ref = p.sum((0, 1))
            tol = ref * (2.2 * score_error(q, k, scale, c.d) + 2.0 ** -17) + TINY * c.g * n
            if accumulate and m > n:
                ref[:m - n] += old[:m - n]
                tol[:m - n] += 2.0 ** -24 * ref[:m - n].abs()
            assert torch.equal(got[m:], old[m:]), (b, h)
            err = (got[:m] - ref).abs()
            assert (err <= tol).all(), (b, h, (err / tol.clamp(min=1e-30)).max())
