"""Paged-cache cases for the tests, and the plain 64-bit form of its operators: one sequence, one
token at a time, on flat tensors (elementary torch operations, no code of the library)."""
from __future__ import annotations

import math

import torch

NAN = float("nan")


def log_f(z):
    """log sigmoid(z) in 64 bits; 0 at +inf."""
    z = z.double()
    return torch.minimum(z, torch.zeros_like(z)) - torch.log1p(torch.exp(-z.abs()))


def rotate(x, cos, sin, pairs):
    """x [n, heads, d] in 64 bits, its first 2 * cos.shape[1] channels turned by the rows' angles."""
    x = x.double().clone()
    half = cos.shape[1]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    cos, sin = cos.double()[:, None], sin.double()[:, None]
    u, w = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    x[..., a], x[..., b] = u, w
    return x


class Case:
    """A pool of pages in no order, filled with NaN, and sequences whose tokens' k, v, z are known.

    own: own tokens of each sequence, the new ones among them (None: an idle sequence).
    new: new tokens of each. prefix: tokens that all share."""

    def __init__(self, own, new, H, Hkv, d, page, dtype="bf16", prefix=0, seed=1, device="cuda", spare=3, tail=0,
                 uniform=False, z_mean=3.0, pages=None):
        self.own, self.new, self.H, self.Hkv, self.d, self.S, self.P = own, new, H, Hkv, d, page, prefix
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype, self.dev, self.B = dtype, torch.device(device), len(own)
        g = self.gen = torch.Generator(self.dev).manual_seed(seed)
        have = [x or 0 for x in own]
        need = [-(-x // page) for x in have]
        npre = -(-prefix // page)
        total = pages if pages is not None else npre + sum(need) + spare
        order = torch.randperm(total, generator=g, device=self.dev)
        order = order[: npre + sum(need)] if pages is None else torch.arange(total - npre - sum(need), total, device=self.dev)
        self.width = max(need + [1])
        self.ptable = order[:npre].to(torch.int32)
        self.table = torch.zeros(self.B, self.width, dtype=torch.int32, device=self.dev)
        at = npre
        for b, n in enumerate(need):
            self.table[b, :n] = order[at : at + n].to(torch.int32)
            at += n
        kw = dict(device=self.dev, dtype=self.dt)
        self.k = torch.empty(total, Hkv, page, d, **kw)
        self.v = torch.empty(total, Hkv, page, d, **kw)
        self.g = torch.full((total, H, page), NAN, device=self.dev)
        self.gbase = torch.full((total, H, 2), NAN, device=self.dev)
        if pages is None:
            self.k.fill_(NAN)
            self.v.fill_(NAN)
        else:  # a pool too large to fill: only what is in use, and around it
            self.k[order], self.v[order] = NAN, NAN
        self.lens = torch.tensor([0 if x is None else x + prefix for x in own], dtype=torch.int32, device=self.dev)
        self.cu = None if uniform else torch.tensor([0] + new, device=self.dev).cumsum(0).to(torch.int32)
        self.rows = sum(new) + tail
        rnd = lambda n, *s: torch.randn(n, *s, generator=g, device=self.dev)  # noqa: E731
        bias = torch.linspace(-1, z_mean + 3, H, device=self.dev)
        seq = lambda n: (rnd(n, Hkv, d).to(self.dt), rnd(n, Hkv, d).to(self.dt), rnd(n, H) + bias)  # noqa: E731
        self.pre, self.seq = seq(prefix), [seq(x) for x in have]
        self.q = rnd(self.rows, H, d).to(self.dt)
        self.row0 = [sum(new[:b]) for b in range(self.B)]

    def put(self, upto_new=True):
        """The tokens held before the call (upto_new: the new ones too) into the pool, by the definition."""
        def one(tok, ids, before, n):
            k, v, z = tok
            c = before + log_f(z).cumsum(0)
            excl = torch.cat([before[None], c[:-1]]) if c.shape[0] else c
            for j0 in range(0, n, self.S):
                m, pg = min(self.S, n - j0), int(ids[j0 // self.S])
                self.k[pg, :, :m] = k[j0 : j0 + m].transpose(0, 1)
                self.v[pg, :, :m] = v[j0 : j0 + m].transpose(0, 1)
                base = excl[j0]
                self.g[pg, :, :m] = (c[j0 : j0 + m] - base).t().float()
                self.gbase[pg, :, 0] = base.float()
                self.gbase[pg, :, 1] = (base - base.float().double()).float()
            return c

        zero = torch.zeros(self.H, dtype=torch.float64, device=self.dev)
        cp = one(self.pre, self.ptable, zero, self.P)
        before = cp[-1] if self.P else zero
        for b in range(self.B):
            if self.own[b] is not None:
                one(self.seq[b], self.table[b], before, self.own[b] - (0 if upto_new else self.new[b]))

    def new_rows(self):
        """k, v, z of the new rows (NaN in rows of idle sequences and behind the last)."""
        k = torch.full((self.rows, self.Hkv, self.d), NAN, device=self.dev, dtype=self.dt)
        v, z = k.clone(), torch.full((self.rows, self.H), NAN, device=self.dev)
        for b in range(self.B):
            if self.own[b] is None or not self.new[b]:
                continue
            for dst, src in zip((k, v, z), self.seq[b]):
                dst[self.row0[b] : self.row0[b] + self.new[b]] = src[self.own[b] - self.new[b] :]
        return k, v, z

    def cache(self, fox):
        return fox.make_cache(self.k, self.v, self.g, self.gbase)

    def batch(self, fox, max_new=None):
        return fox.make_batch(self.lens, self.table, cu_new=self.cu, max_new=max_new or max(self.new + [1]),
                              prefix_table=self.ptable if self.P else None, prefix_len=self.P)

    def attend(self, bias_from_j=False, scale=None, seqs=None):
        """(O, LSE) of all rows in 64 bits; O = 0 and LSE = -inf in idle rows, NaN behind the last."""
        G = self.H // self.Hkv
        scale = self.d**-0.5 if scale is None else scale
        o = torch.full((self.rows, self.H, self.d), NAN, dtype=torch.float64, device=self.dev)
        lse = torch.full((self.rows, self.H), NAN, dtype=torch.float64, device=self.dev)
        for b in range(self.B) if seqs is None else seqs:
            r = slice(self.row0[b], self.row0[b] + self.new[b])
            if self.own[b] is None:
                o[r], lse[r] = 0.0, -math.inf
                continue
            n, N = self.new[b], self.P + self.own[b]
            if not n:
                continue
            k, v, z = (torch.cat([x, y]).double() for x, y in zip(self.pre, self.seq[b]))
            c = log_f(z).cumsum(0)  # [N, H]
            col = torch.cat([torch.zeros_like(c[:1]), c[:-1]]) if bias_from_j else c
            q = self.q[r].double().view(n, self.Hkv, G, self.d)
            x = torch.einsum("nhgd,jhd->hgnj", q, k).reshape(self.H, n, N) * scale
            i = torch.arange(N - n, N, device=self.dev)
            x = x + c[i].t()[:, :, None] - col.t()[:, None]
            x = x.masked_fill(torch.arange(N, device=self.dev) > i[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            w = torch.exp(x - top)
            p = w / w.sum(-1, keepdim=True)
            o[r] = torch.einsum("hgnj,jhd->nhgd", p.view(self.Hkv, G, n, N), v).reshape(n, self.H, self.d)
            lse[r] = (top[..., 0] + w.sum(-1).log()).t()
        return o, lse
