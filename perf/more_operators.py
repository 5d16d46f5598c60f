"""A paged cache held in 4 bits, and the pages themselves: cases, inputs, plain forms and exact values.

append4   new tokens into the 4-bit cache, K (and Q) rotated on the way; then the cache's tokens read back
          as the values that it holds (as before dense attention over them, or a move to another cache)
decode4   attention of the newest tokens of every sequence over the 4-bit cache
step      one step's page bookkeeping: sequences go on, branch, end or begin, and get the pages that they need
compact   the pages in use moved to the front of the pool: which go where, and the tables renamed
copy      pages copied inside a cache, as the two above ask for it

The 4-bit cache, with S tokens a page and blocks of 32 channels of one token and key head:
  value = scale * u, u = -7 .. 7; scale the smallest number of 5 exponent (bias 15) and 3 mantissa bits with
  7 scale >= the block's largest magnitude, and u = x / scale rounded, halves away from zero. A nibble holds u + 8.
  k   [pages, Hkv, S, d / 2]  bytes. 32-bit words [t][block] of a token: channels 8 t .. 8 t + 7 of the block, their
                              nibbles from the lowest in the order 7 2 0 4 6 3 1 5, the word then rotated right by 2 bits
  ks  [pages, Hkv, S, d / 32] scales
  v   [pages, Hkv, S, d / 2]  bytes. 16 bytes a block, two channels a byte, the even one low; block b of slot s stands
                              at place b ^ ((s >> 1) & 3), with two blocks b ^ ((s >> 2) & 1)
  vs  [pages, Hkv, S / 16, 4, d / 32, 4]  scales: token j of 16 at [(j & 7) >> 1][block][2 (j & 1) + (j >> 3)]
  g, gbase                    cumulative log gates: c = gbase[0] + gbase[1] + g
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_NIBBLES = (7, 2, 0, 4, 6, 3, 1, 5)


def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, new=1, H=32, Hkv=8, d=128, page=64, length=1, prefix=0, ragged=False, ragged_new=False,
             rotary="none", rot=0, kind="4bit", pages=0, count=0, mode="none")
    c.update(kw)
    return c


def listed():
    return [
        # a full serving batch's next tokens early in their answers: latency
        _case("append4_batch_step", "append4", B=128, length=64, ragged=True, rotary="half", rot=128),
        # prompts of several users entering the cache, ragged and odd lengths, half of each head rotated in pairs
        _case("append4_prompts", "append4", B=6, new=16384, length=16384, ragged=True, ragged_new=True, rotary="pairs", rot=64),
        # one user, small model, a short odd context: latency
        _case("decode4_short", "decode4", H=16, Hkv=16, d=64, length=1000),
        # one user deep in a long context: the split over keys decides
        _case("decode4_long_context", "decode4", length=65536),
        # a full ragged serving batch: the cache's bandwidth decides
        _case("decode4_batch", "decode4", B=64, length=16384, ragged=True),
        # many questions about one long document
        _case("decode4_shared_document", "decode4", B=256, length=200, prefix=32768, ragged=True),
        # a search with a few hypotheses that branch and end at every step
        _case("step_search", "step", B=8, length=1000, page=16, pages=2048, mode="search"),
        # a serving batch: most sequences go on, some end, some begin with a prompt, some branch
        _case("step_serving", "step", B=512, length=8192, pages=65536, mode="serving", ragged=True),
        # a small pool after some requests ended
        _case("compact_small", "compact", B=16, length=1000, page=16, pages=2048, ragged=True),
        # the pool of a whole card
        _case("compact_large", "compact", B=1024, length=16384, pages=262144, ragged=True, prefix=5000),
        # the partly filled pages of a batch's branches, one layer
        _case("copy_branches", "copy", kind="bf16", count=48, pages=256),
        # a pool of 4-bit pages packed, one layer
        _case("copy_packing", "copy", kind="4bit", count=8192, pages=20000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append4", "decode4", "decode4", "decode4", "step", "compact", "copy"])
    H, Hkv = rng.choice([(16, 16), (32, 8), (32, 32), (12, 4), (14, 2), (8, 1), (16, 8)])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kw = dict(H=H, Hkv=Hkv, d=d, page=page, ragged=rng.random() < 0.7)
    if op == "append4":
        if rng.random() < 0.5:
            B, new = _log_int(rng, 1, 128), rng.randint(1, 4)
            length = max(new, _log_int(rng, 8, 512))
        else:
            B, new = _log_int(rng, 1, 6), _log_int(rng, 5, 4096)
            length = new + rng.randint(0, 500)
            kw["ragged_new"] = rng.random() < 0.5
        kw["rotary"] = rng.choice(["none", "half", "pairs"])
        kw["rot"] = 0 if kw["rotary"] == "none" else rng.choice([d, d // 2])
        kw.update(B=B, new=new, length=length)
    elif op == "decode4" and rng.random() < 0.3:
        B, new = _log_int(rng, 2, 256), rng.choice([1, 1, 2])
        # at most the largest listed case's products, and 64 MB of fp32 scores a head
        most = min(256 * 32 * 32768 // (B * new * H), 16 * 1024 * 1024 * 4 // (B * new))
        kw.update(B=B, new=new, prefix=_log_int(rng, 100, max(200, min(32768, most))), length=max(new, _log_int(rng, 1, 512)))
    elif op == "decode4":
        B, new = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7])
        # at most the largest listed case's keys and values
        most = 64 * 16384 * 8 * 128 // (B * Hkv * d * max(1, new // 2))
        kw.update(B=B, new=new, length=max(new, _log_int(rng, 16, max(32, min(65536, most)))))
        kw["ragged_new"] = new > 1 and rng.random() < 0.5
    elif op == "step":
        B = _log_int(rng, 1, 1024)
        kw.update(B=B, new=rng.choice([1, 1, 5]), length=min(_log_int(rng, 20, 8192), 50000 // B * page), mode=rng.choice(["search", "serving", "go_on"]),
                  prefix=rng.choice([0, 0, 777]))
        kw["pages"] = B * (-(-kw["length"] // page) + 1) + _log_int(rng, 1, 8000)  # sometimes too few
    elif op == "compact":
        kw.update(B=_log_int(rng, 1, 1024), prefix=rng.choice([0, 777]))
        kw["length"] = min(_log_int(rng, 20, 8192), 100000 // kw["B"] * page)
        kw["pages"] = kw["B"] * -(-kw["length"] // page) + 64 + _log_int(rng, 1, 60000)
        kw["count"] = rng.choice([0, 0, _log_int(rng, 1, 1000)])  # at most so many moves
    else:
        kind = rng.choice(["4bit", "4bit", "bf16", "f32"])
        one = Hkv * page * d * 2 * {"4bit": 0.54, "bf16": 2, "f32": 4}[kind] + H * page * 4
        kw.update(kind=kind, count=_log_int(rng, 1, max(2, int(6e8 // one))))
        kw["pages"] = 2 * kw["count"] + rng.randint(1, 100)
    return {k: v for k, v in _case("", op, **kw).items() if k != "name"}


def _counts(case):
    """New tokens and own tokens (the new ones among them) of every sequence."""
    B, new, length = case["B"], case["new"], case["length"]
    n = [1 + (new - 1) * (B - b) // B if case["ragged_new"] else new for b in range(B)]
    # from the full length down to an eighth of it, in steps that are no multiple of a page
    own_len = [length - (b * 7919) % max(1, length * 7 // 8) if case["ragged"] else length for b in range(B)]
    return n, [max(x, y) for x, y in zip(own_len, n)]


def _page_bytes(case):
    """Bytes of one page of a cache of this kind."""
    H, Hkv, d, S = (case[x] for x in ("H", "Hkv", "d", "page"))
    kv = {"4bit": 2 * (d // 2 + d // 32), "bf16": 4 * d, "f32": 8 * d}[case["kind"]]
    return Hkv * S * kv + H * S * 4 + H * 8


def work(case):
    H, Hkv, d, S, B = (case[x] for x in ("H", "Hkv", "d", "page", "B"))
    n, own_len = _counts(case)
    rows, tokens = sum(n), sum(own_len)
    four = 2 * Hkv * (d // 2 + d // 32)  # K and V of a token
    if case["op"] == "append4":
        turned = 2 * rows * H * d * 2 if case["rot"] else 0  # q in and out
        put = rows * (4 * Hkv * d + four + 2 * H * 4 + case["rot"] * 4) + turned
        return {"bytes": put + tokens * (four + 4 * Hkv * d), "flops": 0}
    if case["op"] == "decode4":
        seen = sum(x * (y + case["prefix"]) - x * (x - 1) // 2 for x, y in zip(n, own_len))  # (query, key) pairs a head
        return {"bytes": (tokens + case["prefix"]) * (four + H * 4) + rows * H * (4 * d + 4), "flops": 4 * seen * H * d}
    entries = sum(-(-x // S) for x in own_len)
    if case["op"] == "step":
        return {"bytes": 8 * case["pages"] + 8 * entries + 24 * B, "flops": 0}
    if case["op"] == "compact":
        return {"bytes": 12 * case["pages"] + 8 * entries + 4 * B, "flops": 0}
    return {"bytes": 2 * case["count"] * _page_bytes(case), "flops": 0}


# --------------------------------------------------------------------------------------- the 4-bit form


def _scale_byte(most):
    """Byte of the smallest scale with 7 scale >= most. most / 7 lies at a scale or 2^-9 of it away: fp32 tells, rounded from 64
    bits (a division by a number may be a product with its rounded inverse)."""
    t = (most.double() / 7).float()
    up = ((t.view(torch.int32) + 0xFFFFF) & ~0xFFFFF).view(torch.float32)
    s = torch.where(t >= 2.0**-14, up, torch.ceil(t * 2.0**17) * 2.0**-17).clamp(max=61440.0)
    return ((s.half().view(torch.int16) >> 7) & 0xFF).to(torch.uint8)


def _scale(byte):
    return (byte.to(torch.int16) << 7).view(torch.float16).float()


def _quantise(x):
    """x [..., d] (values of bf16) as codes 1 .. 15 [..., d / 32, 32] and scale bytes [..., d / 32]."""
    x = x.float().unflatten(-1, (-1, 32))
    byte = _scale_byte(x.abs().amax(-1))
    s = _scale(byte)[..., None]
    u = torch.floor(x.abs() / torch.where(s > 0, s, 1.0) + 0.5).clamp(max=7) * torch.sign(x)
    return (u + 8).to(torch.uint8), byte


def _pack_k(code):
    """codes [..., blocks, 32] -> bytes [..., blocks * 16]."""
    w = code.unflatten(-1, (4, 8)).transpose(-3, -2)[..., list(_NIBBLES)].long()  # [..., t, blocks, 8]
    w = (w << torch.arange(0, 32, 4, device=w.device)).sum(-1)
    w = ((w >> 2) | ((w & 3) << 30))
    return ((w[..., None] >> torch.arange(0, 32, 8, device=w.device)) & 255).to(torch.uint8).flatten(-3)


def _unpack_k(data):
    """bytes [..., d / 2] -> codes [..., d / 32, 32]."""
    w = data.view(torch.int32).unflatten(-1, (4, -1))
    w = (w << 2) | ((w >> 30) & 3)
    n = (w[..., None] >> torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)) & 15
    place = torch.tensor([_NIBBLES.index(j) for j in range(8)], device=w.device)
    return n.to(torch.uint8)[..., place].transpose(-3, -2).flatten(-2)


def _places(slot, blocks):
    """Where each block of V in these slots stands: [..., blocks]."""
    turn = (slot >> 1) & 3 if blocks == 4 else (slot >> 2) & 1
    return torch.arange(blocks, device=slot.device) ^ turn[..., None]


def _pack_v(code, slot):
    """codes [n, Hkv, blocks, 32] of tokens in these slots -> bytes [n, Hkv, blocks * 16]."""
    data = code[..., 0::2] | (code[..., 1::2] << 4)
    at = _places(slot, code.shape[-2])[:, None, :, None].expand_as(data)
    return data.gather(-2, at).flatten(-2)  # a place's block is found as a block's place is


def _unpack_v(data):
    """bytes [..., S, d / 2] -> codes [..., S, d / 32, 32]."""
    data = data.unflatten(-1, (-1, 16))
    at = _places(torch.arange(data.shape[-3], device=data.device), data.shape[-2])[..., None].expand_as(data)
    data = data.gather(-2, at)
    return torch.stack([data & 15, data >> 4], -1).flatten(-2)


def _v_scale_at(slot):
    """Where the scale of a token in this slot stands: [S / 16], [4], [4]."""
    j = slot & 15
    return slot >> 4, (j & 7) >> 1, 2 * (j & 1) + (j >> 3)


def _values(k, v, ks, vs):
    """K and V [pages, Hkv, S, d] in fp32 of these pages."""
    a, b, c = _v_scale_at(torch.arange(k.shape[2], device=k.device))
    sv = vs[:, :, a, b, :, c].permute(1, 2, 0, 3)  # [pages, Hkv, S, blocks]
    return tuple(((u.float() - 8) * _scale(s)[..., None]).flatten(-2) for u, s in ((_unpack_k(k), ks), (_unpack_v(v), sv)))


# ------------------------------------------------------------------------------------------- inputs


def _tables(case, dev):
    most = case["prefix"] + max(_counts(case)[1])
    half = case["rot"] // 2
    angle = torch.arange(most, dtype=torch.float64, device=dev)[:, None] * (
        10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half))
    return angle.cos().float(), angle.sin().float()


def _gates(z, before, S):
    """Cumulative log gates of z [n, T, H] (T a multiple of S) after `before` [H], as (local [n, T/S, H, S], base [n, T/S, H, 2])."""
    n, T, H = z.shape
    c = torch.nn.functional.logsigmoid(z.double()).cumsum(1)
    c = c.view(n, T // S, S, H)
    base = torch.cat([torch.zeros_like(c[:, :1, -1]), c[:, :-1, -1]], 1)
    local = (c - base[:, :, None]).permute(0, 1, 3, 2).float()
    base = base + before
    high = base.float()
    return local, torch.stack([high, (base - high.double()).float()], -1)


def _prepare_cache(case, gen, dev):
    B, H, Hkv, d, S, P = (case[x] for x in ("B", "H", "Hkv", "d", "page", "prefix"))
    n, own_len = _counts(case)
    rows, nb, npre = sum(n), -(-max(own_len) // S), -(-P // S)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    # Pages are handed out in no order, some stay free.
    used = [-(-x // S) for x in own_len]
    pages = npre + sum(used) + 3 + B // 4
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    prefix_table = order[:npre].contiguous()
    used_t = torch.tensor(used, device=dev)
    start = npre + used_t.cumsum(0) - used_t
    col = torch.arange(nb, device=dev)
    table = torch.where(col < used_t[:, None], order[(start[:, None] + col).clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    # K and V: unit values, some channels of K several times as large, as after a rotation's slow pairs
    gain = torch.ones(d, device=dev)
    gain[d // 2 - 3 : d // 2] = 4.0
    slot = torch.arange(S, device=dev)
    code, ks = _quantise(normal(pages, Hkv, S, d) * gain)
    k = _pack_k(code)
    code, sv = _quantise(normal(pages, Hkv, S, d))
    v = _pack_v(code.transpose(0, 2).flatten(1, 2), slot).unflatten(1, (Hkv, pages)).permute(2, 1, 0, 3).contiguous()
    a, b, c = _v_scale_at(slot)
    vs = torch.zeros(pages, Hkv, S // 16, 4, d // 32, 4, dtype=torch.uint8, device=dev)
    vs[:, :, a, b, :, c] = sv.permute(2, 0, 1, 3)
    del code, sv
    s = {
        "case": case, "k": k, "v": v, "ks": ks, "vs": vs,
        "g": torch.zeros(pages, H, S, device=dev),
        "gbase": torch.zeros(pages, H, 2, device=dev),
        "table": table,
        "prefix_table": prefix_table if P else None,
        "lens": (torch.tensor(own_len, device=dev) + P).to(torch.int32),  # all tokens, prefix and new ones among them
        "cu": None,
    }
    if case["ragged_new"]:
        s["cu"] = torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)
    # Gate logits: head biases from 0 to 8 (short memories to long ones), unit noise.
    head = torch.linspace(0, 8, H, device=dev)
    before = torch.zeros(H, dtype=torch.float64, device=dev)
    if P:
        z = normal(1, npre * S, H, dtype=torch.float32) + head
        local, base = _gates(z, before, S)
        s["g"][prefix_table.long()], s["gbase"][prefix_table.long()] = local[0], base[0]
        j = P - 1
        before = base[0, j // S].double().sum(-1) + local[0, j // S, :, j % S].double()
    # Tokens that the cache holds before the call: all own ones, or all but the new ones in an append.
    have = torch.tensor([y - x if case["op"] == "append4" else y for x, y in zip(n, own_len)], device=dev)
    if int(have.max()) > 0:
        z = normal(B, nb * S, H, dtype=torch.float32) + head
        local, base = _gates(z, before, S)
        held = (col * S)[None] < have[:, None]
        within = (col[None, :, None] * S + slot) < have[:, None, None]
        local = torch.where(within[:, :, None], local, 0.0)
        at = table.long()[held]
        s["g"][at], s["gbase"][at] = local[held], base[held]
        del z, local, base
    s["q"] = normal(rows, H, d)
    if case["op"] == "append4":
        s["k_new"], s["v_new"] = (normal(rows, Hkv, d) * gain).bfloat16(), normal(rows, Hkv, d)
        s["z"] = normal(rows, H, dtype=torch.float32) + head
        s["cos"], s["sin"] = _tables(case, dev) if case["rot"] else (None, None)
        s["all"] = torch.tensor([0] + own_len, device=dev).cumsum(0).to(torch.int32)
        s["k_all"], s["v_all"] = (torch.zeros(sum(own_len), Hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    if own:  # the handles that a serving loop keeps: they hold the tensors above, and a workspace
        import forget_gated_softmax_gb300 as fox

        s["cache"] = fox.make_cache4(s["k"], s["v"], s["ks"], s["vs"], s["g"], s["gbase"])
        s["batch"] = fox.make_batch(s["lens"], s["table"], cu_new=s["cu"], max_new=case["new"],
                                    prefix_table=s["prefix_table"], prefix_len=P)
        s["ws"] = fox.cache4_workspace(s["cache"], s["batch"], rows)
        if case["op"] == "append4":
            s["whole"] = fox.make_batch(s["lens"], s["table"], cu_new=s["all"], max_new=max(own_len))
    return s


def _prepare_pages(case, gen, dev):
    B, S, P, pages, mode = (case[x] for x in ("B", "page", "prefix", "pages", "mode"))
    _, own_len = _counts(case)
    rand = lambda n: torch.rand(n, generator=gen, device=dev)  # noqa: E731
    i = torch.arange(B, device=dev)
    own_t = torch.tensor(own_len, device=dev)
    # Of every four sequences three are branches of the first, at any of its tokens; of a search all of one.
    root = i - i % (4 if mode != "search" else B)
    common = torch.where(i > root, (rand(B) * torch.minimum(own_t, own_t[root])).long(), 0)
    fresh = (rand(B) < 0.3) & (i > root)  # branches that brought no token of their own yet
    own_t = torch.where(fresh, own_t[root], own_t)
    shared = torch.where(fresh, -(-own_t // S), common // S)
    ended = (rand(B) < 0.05) if mode == "serving" or case["op"] == "compact" else torch.zeros(B, dtype=torch.bool, device=dev)
    ended[0] = False
    lens = torch.where(ended, 0, own_t + P).to(torch.int32)
    width = -(-(case["length"] + 4 * case["new"] + 100) // S)
    npre = -(-P // S)
    col = torch.arange(width, device=dev)
    held = (col < (-(-own_t // S))[:, None]) & ~ended[:, None]
    inherits = held & (col < shared[:, None])
    fresh_page = held & ~inherits
    number = (fresh_page.flatten().cumsum(0) - 1).view(B, width) + npre
    order = torch.randperm(pages, generator=gen, device=dev)
    if case["op"] == "step":  # pages handed out lowest first by a serving loop: mostly at the front
        order = order[(order < pages * 3 // 4).long().argsort(descending=True, stable=True)]
    table = torch.where(fresh_page, order[number.clamp(0, pages - 1)], -1)
    at_root = table[root]
    table = torch.where(inherits, at_root, table).to(torch.int32)
    # a root that had ended is no root: its branches' entries are pages of theirs alone
    missing = held & (table < 0)
    spare = order[(npre + fresh_page.sum() + missing.flatten().cumsum(0) - 1).clamp(0, pages - 1)].view(B, width)
    table = torch.where(missing, spare.to(torch.int32), table).contiguous()
    prefix = order[:npre].to(torch.int32).contiguous()
    refs = torch.bincount(torch.cat([table[held], prefix]).long(), minlength=pages).to(torch.int32)
    s = {"case": case, "refs": refs, "lens": lens, "table": table, "prefix_table": prefix if P else None,
         "refs_out": torch.zeros_like(refs), "table_out": torch.full_like(table, -1)}
    if case["op"] == "step":
        s["lens_out"] = torch.zeros_like(lens)
        s["copies"] = torch.zeros(B, 2, dtype=torch.int32, device=dev)
        s["add"] = torch.full((B,), case["new"], device=dev)
        s["parent"] = None
        if mode == "search":
            s["parent"] = (rand(B) * B).to(torch.int32)
        if mode == "serving":
            x = rand(B)
            parent = torch.where(x < 0.05, (rand(B) * B).long(), i)  # branches
            parent = torch.where((x > 0.95), -1, parent)
            s["add"] = torch.where(x > 0.98, 0, torch.where(x > 0.95, (rand(B) * 90).long() + 1, s["add"]))
            s["parent"] = parent.to(torch.int32)
        s["add"] = s["add"].to(torch.int32)
    else:
        s["prefix_out"] = torch.full_like(prefix, -1) if P else None
        s["map"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["moves"] = torch.zeros(case["count"] or pages // 2, 2, dtype=torch.int32, device=dev)
        s["used"] = torch.zeros(2, dtype=torch.int32, device=dev)
    if own:
        import forget_gated_softmax_gb300 as fox

        now = fox.make_pages(S, s["refs"], s["lens"], s["table"], prefix_table=s["prefix_table"], prefix_len=P)
        out = fox.make_pages(S, s["refs_out"], s.get("lens_out", s["lens"]), s["table_out"], prefix_len=P,
                             prefix_table=s["prefix_table"] if case["op"] == "step" else s["prefix_out"])
        s["pages"], s["out"], s["ws"] = now, out, fox.pages_workspace(now, out)
    return s


def _prepare_copy(case, gen, dev):
    H, Hkv, d, S, pages, count = (case[x] for x in ("H", "Hkv", "d", "page", "pages", "count"))
    s = {"case": case}
    byte = lambda *shape: torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8)  # noqa: E731
    normal = lambda *shape, dtype=torch.float32: torch.randn(*shape, generator=gen, device=dev, dtype=dtype)  # noqa: E731
    if case["kind"] == "4bit":
        s["k"], s["v"] = byte(pages, Hkv, S, d // 2), byte(pages, Hkv, S, d // 2)
        s["ks"], s["vs"] = byte(pages, Hkv, S, d // 32), byte(pages, Hkv, S // 16, 4, d // 32, 4)
    else:
        s["k"], s["v"] = (normal(pages, Hkv, S, d, dtype=_DTYPES[case["kind"]]) for _ in range(2))
    s["g"], s["gbase"] = normal(pages, H, S), normal(pages, H, 2)
    order = torch.randperm(pages, generator=gen, device=dev)
    pairs = torch.stack([order[:count], order[count : 2 * count]], 1).to(torch.int32)
    none = torch.full((count // 8 + 1, 2), -1, dtype=torch.int32, device=dev)  # sequences that copy nothing
    s["pairs"] = torch.cat([none, pairs])[torch.randperm(pairs.shape[0] + none.shape[0], generator=gen, device=dev)].contiguous()
    if own:
        import forget_gated_softmax_gb300 as fox

        s["cache"] = (fox.make_cache4(s["k"], s["v"], s["ks"], s["vs"], s["g"], s["gbase"]) if case["kind"] == "4bit" else
                      fox.make_cache(s["k"], s["v"], s["g"], s["gbase"]))
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    if case["op"] in ("append4", "decode4"):
        return _prepare_cache(case, gen, dev)
    return _prepare_copy(case, gen, dev) if case["op"] == "copy" else _prepare_pages(case, gen, dev)


# ------------------------------------------------------------------------------------------- a pass


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import forget_gated_softmax_gb300 as fox

        if op == "append4":
            turned = fox.fox_cache4_append(s["cache"], s["batch"], s["k_new"], s["v_new"], s["z"],
                                           q=s["q"] if case["rot"] else None, cos=s["cos"], sin=s["sin"],
                                           pairs=case["rotary"] == "pairs", ws=s["ws"])
            k, v = fox.fox_cache4_read(s["cache"], s["whole"], k=s["k_all"], v=s["v_all"], ws=s["ws"])
            return k, v, s["g"], s["gbase"], turned
        if op == "decode4":
            return fox.fox_cache4_decode(s["cache"], s["batch"], s["q"], ws=s["ws"])
        if op == "step":
            fox.fox_pages_step(s["pages"], s["add"], s["copies"], parent=s["parent"], out=s["out"], ws=s["ws"])
            return s["lens_out"], s["table_out"], s["refs_out"], s["copies"]
        if op == "compact":
            fox.fox_pages_compact(s["pages"], s["map"], s["moves"], s["used"], out=s["out"], ws=s["ws"])
            return s["table_out"], s["prefix_out"], s["refs_out"], s["map"], s["moves"], s["used"]
        fox.fox_cache_copy(s["cache"], s["pairs"], ws=s["ws"])
        return [s[x] for x in ("k", "v", "ks", "vs", "g", "gbase") if x in s]
    return {"append4": _append, "decode4": _attend, "step": _step, "compact": _compact, "copy": _copy}[op](s)


# ------------------------------------------------------------------------------------- plain forms


def _rows(s, cu, rows):
    """Sequence and position of every row; cu: first row of each sequence, or None: the same number each."""
    i = torch.arange(rows, device=s["q"].device)
    if cu is None:
        each = rows // s["lens"].numel()
        b = i // each
        return b, s["lens"][b].long() - each + i % each
    cu = cu.long()
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, s["lens"][b].long() - (cu[b + 1] - i)


def _nearest_bf16(x):
    """x in 64 bits to bf16, rounded once: an fp32 that lies halfway is first moved to the side that x is on."""
    f = x.float()
    rest = x - f.double()
    halfway = (f.view(torch.int32) & 0xFFFF) == 0x8000
    way = torch.where(rest > 0, math.inf, -math.inf).float()
    return torch.where(halfway & (rest != 0), torch.nextafter(f, way), f).bfloat16()


def _turn(x, cos, sin, pairs):
    """x [rows, heads, d] with its first 2 * cos.shape[1] channels rotated by the rows' angles. In 64 bits: a rounding to
    the other side of a border would be a whole step of the 4-bit form."""
    r = cos.shape[1] * 2
    cos, sin = cos[:, None].double(), sin[:, None].double()
    a, b = (x[..., 0:r:2].double(), x[..., 1:r:2].double()) if pairs else (x[..., : r // 2].double(), x[..., r // 2 : r].double())
    u, w = _nearest_bf16(a * cos - b * sin), _nearest_bf16(b * cos + a * sin)
    turned = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _append(s):
    case, S = s["case"], s["case"]["page"]
    b, pos = _rows(s, s["cu"], s["q"].shape[0])
    page, slot = s["table"][b, pos // S].long(), pos % S
    k, q = s["k_new"], None
    if case["rot"]:
        cos, sin = s["cos"][pos], s["sin"][pos]
        k = _turn(k, cos, sin, case["rotary"] == "pairs")
        q = _turn(s["q"], cos, sin, case["rotary"] == "pairs")
    code, scale = _quantise(k)
    s["k"][page, :, slot] = _pack_k(code)
    s["ks"][page, :, slot] = scale
    code, scale = _quantise(s["v_new"])
    s["v"][page, :, slot] = _pack_v(code, slot)
    a, t, e = _v_scale_at(slot)
    s["vs"][page, :, a, t, :, e] = scale
    # Gates: the running sum goes on from the token before the sequence's first new one.
    rows = pos.numel()
    first = torch.searchsorted(b, b)  # row of the sequence's first new token
    a = -torch.log1p(torch.exp(-s["z"].double().abs())) + s["z"].double().clamp(max=0)
    total = a.cumsum(0)
    since = total - total[first] + a[first]
    p0 = pos[first] - 1
    pg = s["table"][b, p0.clamp(min=0) // S].long()
    was = s["gbase"][pg].double().sum(-1) + s["g"][pg, :, p0.clamp(min=0) % S].double()
    c = since + torch.where((p0 >= 0)[:, None], was, 0.0)
    # A page's base: the sum before its first token, kept where the page had begun before the call.
    opens = torch.arange(rows, device=pos.device) - slot  # row of the page's first token, if it is a new one
    begun = opens >= first
    o = torch.maximum(opens, first)
    base = torch.where(begun[:, None], c[o] - a[o], s["gbase"][page].double().sum(-1))
    high = base.float()
    s["g"][page, :, slot] = (c - base).float()
    low = (base - high.double()).float()
    s["gbase"][page[begun]] = torch.stack([high, low], -1)[begun]
    # What the cache then holds of every sequence.
    b, pos = _rows(s, s["all"], s["k_all"].shape[0])
    page, slot = s["table"][b, pos // S].long(), pos % S
    a, t, e = _v_scale_at(slot)
    code = _unpack_k(s["k"][page, :, slot])
    s["k_all"].copy_(((code.float() - 8) * _scale(s["ks"][page, :, slot])[..., None]).flatten(-2))
    data = s["v"][page, :, slot].unflatten(-1, (-1, 16))
    data = data.gather(-2, _places(slot, data.shape[-2])[:, None, :, None].expand_as(data))
    code = torch.stack([data & 15, data >> 4], -1).flatten(-2)
    s["v_all"].copy_(((code.float() - 8) * _scale(s["vs"][page, :, a, t, :, e])[..., None]).flatten(-2))
    return s["k_all"], s["v_all"], s["g"], s["gbase"], q


def _attend(s):
    case = s["case"]
    H, Hkv, d, S, P, B = (case[x] for x in ("H", "Hkv", "d", "page", "prefix", "B"))
    G = H // Hkv
    b, pos = _rows(s, s["cu"], s["q"].shape[0])
    t = pos - s["lens"][b].long() + case["new"]  # place in a padded [B, new] batch of rows
    dev = pos.device
    q = torch.zeros(B, case["new"], H, d, device=dev)
    q[b, t] = s["q"].float() / math.sqrt(d)
    q = q.view(B, -1, Hkv, G, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, new, d]
    key, val = _values(s["k"], s["v"], s["ks"], s["vs"])
    table = s["table"].long()
    keys = torch.arange(table.shape[1] * S, device=dev)
    cum = s["gbase"][table].double().sum(-1)[..., None] + s["g"][table].double()  # [B, pages, H, S]
    cum = cum.permute(0, 2, 1, 3).reshape(B, H, -1)
    at = (s["lens"].long()[:, None] - case["new"] + torch.arange(case["new"], device=dev) - P)  # own place of the rows
    ci = cum.gather(2, at.clamp(min=0)[:, None].expand(-1, H, -1))
    bias = (ci[..., None] - cum[:, :, None]).float()
    bias = torch.where(keys <= at[:, None, :, None], bias, -math.inf)  # [B, H, new, keys]
    k = key[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, -1, d)
    score = (q @ k.transpose(-1, -2)).view(B, H, case["new"], -1) + bias
    del k, bias
    if P:
        pt = s["prefix_table"].long()
        kp = key[pt].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :P]
        vp = val[pt].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :P]
        cp = (s["gbase"][pt].double().sum(-1)[..., None] + s["g"][pt].double()).permute(1, 0, 2).reshape(H, -1)[:, :P]
        tall = q.permute(1, 2, 0, 3, 4).reshape(Hkv, -1, d)  # all rows of a key head against the one prefix
        sp = (tall @ kp.transpose(-1, -2)).view(H, B, case["new"], P)
        # c_i - c_j = (c_i - c_last) + (c_last - c_j), c_last the prefix's last token's
        sp = sp + (cp[:, -1:] - cp).float()[:, None, None] + (ci.permute(1, 0, 2) - cp[:, -1, None, None]).float()[..., None]
        most = torch.maximum(score.amax(-1), sp.amax(-1).permute(1, 0, 2))
        sp = torch.exp(sp - most.permute(1, 0, 2)[..., None])
    else:
        most = score.amax(-1)
    del key
    w = torch.exp(score - torch.where(torch.isfinite(most), most, 0.0)[..., None])
    total = w.sum(-1)
    v = val[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, -1, d)
    v = torch.where((keys < (s["lens"].long() - P)[:, None])[:, None, None, :, None], v, 0.0)
    o = (w.view(B, Hkv, G, case["new"], -1) @ v).view(B, H, case["new"], d)
    if P:
        total = total + sp.sum(-1).permute(1, 0, 2)
        op = (sp.reshape(Hkv, -1, P) @ vp).view(H, B, case["new"], d)
        o = o + op.permute(1, 0, 2, 3)
    o, lse = o / total[..., None], most + torch.log(total)
    return o.permute(0, 2, 1, 3)[b, t].to(s["q"].dtype), lse.permute(0, 2, 1)[b, t].contiguous()


def _held(lens, table, S, P):
    """Entries of the tables that name a page of the sequence's."""
    count = -(-(lens.long() - P).clamp(min=0) // S)
    return torch.arange(table.shape[1], device=table.device) < count[:, None]


def _step(s):
    case = s["case"]
    S, P, B = case["page"], case["prefix"], case["B"]
    lens, table, add = s["lens"].long(), s["table"], s["add"].long()
    dev = lens.device
    parent = torch.arange(B, device=dev) if s["parent"] is None else s["parent"].long()
    # References: each old sequence's pages gain its children and lose the sequence itself.
    kids = torch.zeros(B, dtype=torch.int32, device=dev)
    kids.index_add_(0, parent.clamp(min=0), (parent >= 0).to(torch.int32))
    held = _held(lens, table, S, P)
    refs = s["refs_out"].copy_(s["refs"])
    refs.index_add_(0, table[held].long(), (kids - 1)[:, None].expand_as(table)[held])
    # What the new sequences begin with, and need.
    src = parent.clamp(min=0)
    length = torch.where(parent >= 0, lens[src], 0)
    have = (length - P).clamp(min=0)
    grows = (add > 0) & (have + add <= table.shape[1] * S)
    n0, n1 = -(-have // S), -(-(have + add) // S)
    last = table[src, (n0 - 1).clamp(min=0)].long()
    part = grows & (have % S > 0)
    before = ((last[:, None] == last) & part & torch.ones(B, B, dtype=torch.bool, device=dev).tril(-1)).sum(1)
    copied = part & (refs[last.clamp(min=0)] - before > 1)
    need = torch.where(grows, n1 - n0 + copied, 0)
    upto = need.cumsum(0)
    free = torch.cat([(refs <= 0).nonzero().flatten(), torch.zeros(1, dtype=torch.long, device=dev)])
    grows = grows & ((need == 0) | (upto <= free.numel() - 1))
    copied = copied & grows
    at = upto - need
    # Tables: the parent's pages, the copied last one, new ones.
    col = torch.arange(table.shape[1], device=dev)
    first = (at + copied - n0)[:, None] + col
    page = torch.where(col < n0[:, None], table[src].long(), free[first.clamp(0, free.numel() - 1)])
    fresh = free[at.clamp(max=free.numel() - 1)]
    page = torch.where(copied[:, None] & (col == (n0 - 1)[:, None]), fresh[:, None], page)
    new = grows[:, None] & (col >= n0[:, None]) & (col < n1[:, None])
    s["table_out"].copy_(torch.where(new | (col < n0[:, None]), page, s["table_out"]))
    refs[page[new]] = 1
    refs.index_add_(0, last[copied], torch.full_like(last[copied], -1, dtype=torch.int32))
    refs[fresh[copied]] = 1
    s["copies"].copy_(torch.where(copied[:, None], torch.stack([last, fresh], 1), -1))
    s["lens_out"].copy_(torch.where(grows, torch.where(length > 0, length, P) + add, length))
    return s["lens_out"], s["table_out"], refs, s["copies"]


def _compact(s):
    case = s["case"]
    refs = s["refs"]
    i = torch.arange(refs.numel(), device=refs.device)
    used = (refs > 0).sum()
    source = ((refs > 0) & (i >= used)).nonzero().flatten().flip(0)[: s["moves"].shape[0]]
    to = ((refs <= 0) & (i < used)).nonzero().flatten()[: source.numel()]
    renamed = s["map"].copy_(i)
    renamed[source] = to.to(torch.int32)
    moves = s["moves"].fill_(-1)
    moves[: source.numel()] = torch.stack([source, to], 1).to(torch.int32)
    out = s["refs_out"].copy_(refs)
    out[to], out[source] = refs[source], 0
    held = _held(s["lens"], s["table"], case["page"], case["prefix"])
    s["table_out"].copy_(torch.where(held, renamed[torch.where(held, s["table"], 0).long()], s["table_out"]))
    if case["prefix"]:
        s["prefix_out"].copy_(renamed[s["prefix_table"].long()])
    s["used"].copy_(torch.stack([used, torch.where(out > 0, i + 1, 0).amax()]))
    return s["table_out"], s["prefix_out"], out, renamed, moves, s["used"]


def _copy(s):
    pairs = s["pairs"].long()
    pairs = pairs[pairs[:, 0] >= 0]
    arrays = [s[x] for x in ("k", "v", "ks", "vs", "g", "gbase") if x in s]
    return [x.index_copy_(0, pairs[:, 1], x[pairs[:, 0]]) for x in arrays]


# ------------------------------------------------------------------------------------ exact values


def _exact_power(e):
    """2^e in 64 bits, bit for bit (pow need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_scale(byte):
    e, m = byte.long() // 8, byte.long() % 8
    return torch.where(e > 0, (8 + m) * _exact_power(e - 18), m * _exact_power(e * 0 - 17))


def _exact_values(s, pages):
    """K and V of these pages [pages, Hkv, S, d] in 64 bits, bit by bit as the layout is described."""
    d, S, blocks = s["case"]["d"], s["case"]["page"], s["case"]["d"] // 32
    dev = s["k"].device
    ch, slot = torch.arange(d, device=dev), torch.arange(S, device=dev)
    b, r = ch // 32, ch % 32
    nibble = torch.tensor(_NIBBLES, device=dev).argsort()[r % 8]
    k = s["k"][pages]
    u = torch.zeros(*k.shape[:3], d, dtype=torch.float64, device=dev)
    for i in range(4):  # bit i of the nibble, after the rotation
        bit = (4 * nibble + i - 2) % 32
        u += 2.0**i * ((k[..., ((r // 8) * blocks + b) * 4 + bit // 8] >> (bit % 8).to(torch.uint8)) & 1)
    key = (u - 8) * _exact_scale(s["ks"][pages])[..., b]
    turn = (slot // 2) % 4 if blocks == 4 else (slot // 4) % 2
    place = torch.bitwise_xor(b[None], turn[:, None]) * 16 + r // 2  # [S, d]
    data = s["v"][pages][:, :, slot[:, None], place]
    u = torch.where(ch % 2 == 0, data % 16, data // 16).double()
    j = slot % 16
    scale = s["vs"][pages][:, :, (slot // 16)[:, None], ((j % 8) // 2)[:, None], b[None], (2 * (j % 2) + j // 8)[:, None]]
    return key, (u - 8) * _exact_scale(scale)


def _exact_hold(x):
    """x [..., d] in 64 bits as the 4-bit form holds it."""
    y = x.unflatten(-1, (-1, 32))
    most = y.abs().amax(-1, keepdim=True)
    t = most / torch.full_like(most, 7.0)
    # the quantum of a number of 4 significant bits
    q = _exact_power(torch.clamp(torch.frexp(t)[1] - 4, min=-17))
    s = torch.ceil(t / q) * q
    return (torch.sign(y) * torch.floor(y.abs() / s.clamp(min=2.0**-17) + 0.5) * s).flatten(-2)


def _exact_bf16(x):
    m, e = torch.frexp(x)
    return torch.round(m * 256) / 256 * _exact_power(e)


def exact(case, seed):
    """The definition, one sequence after the other, in 64 bits. What the pages' operators return are whole numbers and copies."""
    if case["op"] not in ("append4", "decode4"):
        return None
    s = prepare(case, seed)
    n, own_len = _counts(case)
    H, Hkv, d, S, P = (case[x] for x in ("H", "Hkv", "d", "page", "prefix"))
    dev = s["q"].device
    logf = lambda z: torch.nn.functional.logsigmoid(z.double())  # noqa: E731
    row = 0
    if case["op"] == "append4":
        g, gb = s["g"].double(), s["gbase"].double()
        turned = torch.empty(sum(n), H, d, dtype=torch.float64, device=dev) if case["rot"] else None
        ks, vs = [], []
        for b, (new, length) in enumerate(zip(n, own_len)):
            ids = s["table"][b, : -(-length // S)].long()
            k, v = (x.transpose(1, 2).flatten(0, 1)[:length] for x in _exact_values(s, ids))
            here = torch.arange(length - new, length, device=dev)
            page, slot = s["table"][b].long()[here // S], here % S
            kn, qn = s["k_new"][row : row + new].double(), s["q"][row : row + new].double()
            if case["rot"]:
                half = case["rot"] // 2
                turn = torch.complex(s["cos"].double(), s["sin"].double())[here][:, None]
                for x in (kn, qn):
                    i = torch.arange(half, device=dev)
                    re, im = (2 * i, 2 * i + 1) if case["rotary"] == "pairs" else (i, i + half)
                    y = torch.complex(x[..., re], x[..., im]) * turn
                    x[..., re], x[..., im] = y.real, y.imag
                kn = _exact_bf16(kn)
                turned[row : row + new] = qn
            k[here], v[here] = _exact_hold(kn), _exact_hold(s["v_new"][row : row + new].double())
            ks.append(k)
            vs.append(v)
            c = torch.zeros(H, dtype=torch.float64, device=dev)
            if length > new:
                p = length - new - 1
                c = gb[s["table"][b, p // S].long()].sum(-1) + g[s["table"][b, p // S].long(), :, p % S]
            c = c + torch.cumsum(logf(s["z"][row : row + new]), 0)  # of the new tokens
            opening = (slot == 0).nonzero().flatten()
            before = c[opening] - logf(s["z"][row : row + new])[opening]
            gb[page[opening], :, 0] = before.float().double()
            gb[page[opening], :, 1] = before - before.float().double()
            g[page, :, slot] = c - gb[page].sum(-1)
            row += new
        return torch.cat(ks), torch.cat(vs), g, gb, turned
    o = torch.empty(sum(n), H, d, dtype=torch.float64, device=dev)
    lse = torch.empty(sum(n), H, dtype=torch.float64, device=dev)
    flat = lambda x: x.transpose(0, 1).flatten(1, 2)  # noqa: E731  [pages, heads, S, ...] -> [heads, tokens, ...]
    if P:
        pt = s["prefix_table"].long()
        pre = [flat(x)[:, :P] for x in (*_exact_values(s, pt), s["gbase"][pt].double().sum(-1)[..., None] + s["g"][pt].double())]
    for b, (new, length) in enumerate(zip(n, own_len)):
        ids = s["table"][b, : -(-length // S)].long()
        key, val = (flat(x)[:, :length] for x in _exact_values(s, ids))
        c = flat(s["gbase"][ids].double().sum(-1)[..., None] + s["g"][ids].double())[:, :length]
        if P:
            key, val, c = (torch.cat([x, y], 1) for x, y in zip(pre, (key, val, c)))
        qb = s["q"][row : row + new].double().transpose(0, 1)  # [H, new, d]
        x = torch.matmul(qb.reshape(Hkv, -1, d), key.transpose(1, 2)).view(H, new, -1) / d**0.5
        i = torch.arange(P + length - new, P + length, device=dev)
        x = x + c[:, i][:, :, None] - c[:, None]
        x = x.masked_fill(torch.arange(P + length, device=dev) > i[:, None], -math.inf)
        l = torch.logsumexp(x, -1)
        p = torch.exp(x - l[..., None])
        o[row : row + new] = torch.matmul(p.view(Hkv, -1, P + length), val).view(H, new, d).transpose(0, 1)
        lse[row : row + new] = l.t()
        row += new
    return o, lse
