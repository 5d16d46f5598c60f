"""The 4-bit cache for the tests: what a block of values is held as, in 64 bits and by search rather than by arithmetic, and
its bytes, written place by place as include/fox.h describes them. No code of the library."""
from __future__ import annotations

import torch

from cachetest import Case

SCALES = [m * 2.0**-17 if e == 0 else (8 + m) * 2.0 ** (e - 18) for e in range(31) for m in range(8)]  # by byte
NIBBLES = [7, 2, 0, 4, 6, 3, 1, 5]


def nearest_bf16(x):
    """x in 64 bits to the nearest bf16 (ties to even), as bf16 and by one rounding: to 8 significant bits first."""
    m, e = torch.frexp(x)
    power = ((e.long() + 1023) << 52).view(torch.float64)
    return (torch.round(m * 256) / 256 * power).to(torch.bfloat16)


def hold(x):
    """x [..., d] (finite, at most 430080) as (u [..., d] in -7 .. 7, scale bytes [..., d / 32], values [..., d]) in 64 bits."""
    y = x.double().unflatten(-1, (-1, 32))
    table = torch.tensor(SCALES, dtype=torch.float64, device=x.device)
    most = y.abs().amax(-1)
    byte = torch.searchsorted(7 * table, most.contiguous())  # the first with 7 s >= most
    s = table[byte][..., None]
    steps = torch.arange(8, dtype=torch.float64, device=x.device)
    # the least u whose upper border (u + 1/2) s lies above |y|: halves away from zero
    u = (y.abs()[..., None] >= (steps[:7] + 0.5) * s[..., None]).sum(-1).double()
    u = torch.where(s > 0, u, 0.0) * torch.sign(y)
    return u.flatten(-2), byte, (u * s).flatten(-2)


def k_bits(d):
    """Bit of a token's row of k at which bit 0 .. 3 of each channel's nibble stands: [d, 4]."""
    at = torch.empty(d, 4, dtype=torch.long)
    for c in range(d):
        b, t, j = c // 32, c % 32 // 8, c % 8
        for i in range(4):
            at[c, i] = (t * (d // 32) + b) * 32 + (4 * NIBBLES.index(j) + i - 2) % 32
    return at


def v_bits(d, slot):
    at = torch.empty(d, 4, dtype=torch.long)
    for c in range(d):
        place = (c // 32) ^ (slot // 2 % 4 if d == 128 else slot // 4 % 2)
        for i in range(4):
            at[c, i] = place * 128 + c % 32 * 4 + i
    return at


def v_scale_place(slot, block, blocks):
    j = slot % 16
    return slot // 16 * 16 * blocks + (j % 8 // 2) * 4 * blocks + block * 4 + 2 * (j % 2) + j // 8


def row_bytes(u, bits):
    """u [n, heads, d] as rows of d / 2 bytes, by the places of the bits ([n, d, 4] or [d, 4])."""
    code = (u.long() + 8)[..., None] >> torch.arange(4, device=u.device) & 1  # [n, heads, d, 4]
    n, heads, d, _ = code.shape
    bits = bits.to(u.device).expand(n, d, 4)[:, None].expand(n, heads, d, 4)
    flat = torch.zeros(n, heads, d * 4, dtype=torch.long, device=u.device)
    flat.scatter_(2, bits.flatten(2), code.flatten(2))
    return (flat.unflatten(2, (-1, 8)) << torch.arange(8, device=u.device)).sum(-1).to(torch.uint8)


class Case4(Case):
    """A Case whose pool is held in 4 bits, everything that nothing was put into all ones (scales of NaN)."""

    def __init__(self, *a, low=False, **kw):
        super().__init__(*a, **kw)
        pages = self.k.shape[0]
        byte = lambda *s: torch.full(s, 255, dtype=torch.uint8, device=self.dev)  # noqa: E731
        if kw.get("pages") is not None:
            byte = lambda *s: torch.empty(s, dtype=torch.uint8, device=self.dev)  # noqa: E731
        S, d, Hkv = self.S, self.d, self.Hkv
        self.k4, self.v4 = byte(pages, Hkv, S, d // 2), byte(pages, Hkv, S, d // 2)
        self.ks, self.vs = byte(pages, Hkv, S, d // 32), byte(pages, Hkv, S // 16, 4, d // 32, 4)
        self.g_low = torch.full_like(self.g, float("nan")) if low else None
        self.kbits = k_bits(d)
        self.vbits = torch.stack([v_bits(d, s) for s in range(S)])
        self.held = {}  # sequence (-1: the prefix) -> K, V values [tokens, Hkv, d] in 64 bits

    def put4(self, ids, j0, k, v):
        """Tokens j0 .. of a sequence whose pages are `ids`, into the pool; returns their values."""
        n, blocks = k.shape[0], self.d // 32
        if n == 0:
            return k.double(), v.double()
        j = torch.arange(j0, j0 + n, device=self.dev)
        page, slot = ids.long()[j // self.S], j % self.S
        uk, bk, kv = hold(k)
        uv, bv, vv = hold(v)
        self.k4[page, :, slot] = row_bytes(uk, self.kbits)
        self.v4[page, :, slot] = row_bytes(uv, self.vbits[slot.cpu()])
        self.ks[page, :, slot] = bk.to(torch.uint8)
        places = torch.tensor([[v_scale_place(s, b, blocks) for b in range(blocks)] for s in range(self.S)], device=self.dev)
        flat = self.vs.view(self.vs.shape[0], self.Hkv, -1)
        for b in range(blocks):
            flat[page, :, places[slot, b]] = bv[..., b].to(torch.uint8)
        return kv, vv

    def put(self, upto_new=True, turn=None):
        """As Case.put, K and V in 4 bits; `turn(k, first position)` rotates K rows before they are held."""
        super().put(upto_new)
        turn = turn or (lambda k, at: k)
        self.held[-1] = self.put4(self.ptable, 0, turn(self.pre[0], 0), self.pre[1])
        for b in range(self.B):
            if self.own[b] is None:
                continue
            n = self.own[b] - (0 if upto_new else self.new[b])
            self.held[b] = self.put4(self.table[b], 0, turn(self.seq[b][0][:n], self.P), self.seq[b][1][:n])

    def cache4(self, fox):
        return fox.make_cache4(self.k4, self.v4, self.ks, self.vs, self.g, self.gbase, self.g_low)

    def attend(self, **kw):
        """Case.attend over the values that the cache holds."""
        pre, seq = self.pre, self.seq
        self.pre = (*self.held[-1], pre[2])
        self.seq = [(*self.held[b], x[2]) if b in self.held else x for b, x in enumerate(seq)]
        try:
            return super().attend(**kw)
        finally:
            self.pre, self.seq = pre, seq
