"""Paged-cache inputs and the plain fp64 definitions the paged operators are tested against."""
import math

import numpy as np
import torch

from oracle import attention_fwd

EPS_BF16 = 2.0 ** -8   # half a step of bf16, relative (rounding to nearest)
EPS_F32 = 2.0 ** -24


def to64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Cache:
    """A pool of pages in either order, tables over a random permutation of its pages."""

    def __init__(self, lens, hkv, page, d, seed=0, prefix=0, rows_first=False, spare=3, width_extra=0, one_tensor=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.page, self.d, self.prefix = list(lens), hkv, page, d, prefix
        need = [-(-n // page) for n in lens]
        n_pre = -(-prefix // page)
        self.pages = sum(need) + n_pre + spare
        shape = (self.pages, page, hkv, d) if rows_first else (self.pages, hkv, page, d)
        if one_tensor:  # keys and values of a page side by side in one tensor
            both = torch.randn((shape[0], 2, *shape[1:]), generator=g).to(torch.bfloat16).cuda()
            k, v = both[:, 0], both[:, 1]
        else:
            k = torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
            v = torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
        self.k = k.permute(0, 2, 1, 3) if rows_first else k
        self.v = v.permute(0, 2, 1, 3) if rows_first else v
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.prefix_pages = perm[:n_pre].cuda()
        # entries past a sequence's last page name no page at all
        t = torch.full((len(lens), max([1] + need) + width_extra), -7, dtype=torch.int32)
        at = n_pre
        for b, n in enumerate(need):
            t[b, :n] = perm[at:at + n]
            at += n
        self.used = set(perm[:at].tolist())
        self.tables = t.cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()

    def poison(self):
        """NaN wherever no key of the batch lives: unused pages and the rows behind the last keys."""
        for p in set(range(self.pages)) - self.used:
            self.k[p] = math.nan
            self.v[p] = math.nan
        for b, n in enumerate(self.lens):
            if n % self.page:
                p = int(self.tables[b, n // self.page])
                self.k[p, :, n % self.page:] = math.nan
                self.v[p, :, n % self.page:] = math.inf
        if self.prefix % self.page:
            p = int(self.prefix_pages[-1])
            self.k[p, :, self.prefix % self.page:] = math.nan
            self.v[p, :, self.prefix % self.page:] = -math.inf

    def _gather(self, pool, table, n, h):
        p64 = [to64(pool[int(p), h]) for p in table[: -(-n // self.page)]]
        return np.concatenate(p64)[:n] if p64 else np.zeros((0, self.d))

    def keys_values(self, b, h):
        t, n = self.tables[b].tolist(), self.lens[b]
        k, v = self._gather(self.k, t, n, h), self._gather(self.v, t, n, h)
        if self.prefix:
            t = self.prefix_pages.tolist()
            k = np.concatenate([self._gather(self.k, t, self.prefix, h), k])
            v = np.concatenate([self._gather(self.v, t, self.prefix, h), v])
        return k, v


def check_decode(c, q, o, lse, scale, heads=None, seqs=None):
    """Every row of o and lse against the definition.

    Bounds: o is rounded to bf16 once (half a step of |o|); every weight of the
    P V product is rounded to bf16 once, which moves o by at most half a step of
    sum_j p_j |v_j|; a score is a sum of d products in fp32, off by at most
    e = (d + 8) 2^-24 scale sum |q k| (any order of summation), the exponential
    and the merge of partial results add 2^-19 relative, and both enter the
    numerator and the denominator.
    """
    B, hq, nq, d = q.shape
    g = hq // c.hkv
    q64, o64, l64 = to64(q), to64(o), to64(lse)
    for b in range(B) if seqs is None else seqs:
        for h in range(c.hkv) if heads is None else heads:
            k, v = c.keys_values(b, h)
            for i in range(nq):
                n = c.prefix + max(0, c.lens[b] - nq + 1 + i)
                for hh in range(h * g, (h + 1) * g):
                    if n == 0:
                        assert (o64[b, hh, i] == 0).all() and l64[b, hh, i] == -np.inf, (b, hh, i)
                        continue
                    qr = q64[b, hh, i][None]
                    ref, L = attention_fwd(qr, k[:n], v[:n], scale)
                    a, _ = attention_fwd(qr, k[:n], np.abs(v[:n]), scale)
                    e = (d + 8) * EPS_F32 * scale * (np.abs(k[:n]) @ np.abs(qr[0])).max() + 2.0 ** -19
                    tol = EPS_BF16 * np.abs(ref[0]) + (1.01 * EPS_BF16 + 2 * e) * a[0]
                    err = np.abs(o64[b, hh, i] - ref[0])
                    assert np.isfinite(o64[b, hh, i]).all() and (err <= tol).all(), (b, hh, i, n, (err / tol).max())
                    assert abs(l64[b, hh, i] - L[0]) <= e + abs(L[0]) * 2.0 ** -22 + 2.0 ** -19, (b, hh, i, n, l64[b, hh, i], L[0])


def rotate64(x, cos, sin, interleaved):
    """Rows of heads [..., d] rotated by one position's cosines and sines, in fp64, and the
    sizes |a c| + |b s| of what is summed."""
    half = cos.shape[-1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, size = x.copy(), np.abs(x)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    size[..., a] = np.abs(x[..., a] * cos) + np.abs(x[..., b] * sin)
    size[..., b] = np.abs(x[..., a] * sin) + np.abs(x[..., b] * cos)
    return y, size


def check_rotated(got, x, cos, sin, interleaved, where):
    """Three fp32 roundings of the summands' sizes, then one to bf16; elements past the rotated ones are copies."""
    y, size = rotate64(x, cos, sin, interleaved)
    tol = EPS_BF16 * np.abs(y) * (1 + 2.0 ** -8) + 4 * EPS_F32 * size
    rot = 2 * cos.shape[-1]
    assert (got[..., rot:] == x[..., rot:]).all(), where
    assert (np.abs(got - y) <= tol)[..., :rot].all(), where
