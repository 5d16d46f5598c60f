"""The paged-cache operators of forget-gated attention: cases, inputs, plain forms and exact values.

Three operators, as a serving loop calls them once a layer and step:

append  new tokens' K, V and gate logits z into a paged cache, K (and Q) rotated on the way
decode  attention of the newest tokens of every sequence over its pages
shared  the same for a batch whose sequences share a long prefix (a system prompt, a
        document, the root of a search), computed once for all

The cache, with S tokens a page:
  k, v   [pages, Hkv, S, d]
  g      [pages, H, S]     sum of log sigmoid(z) from the page's first token to this one
  gbase  [pages, H, 2]     the sum over every token before the page, as two fp32 (high, low)
so that the cumulative log gate of a token is c = gbase[0] + gbase[1] + g, and the bias of
key j for query i is c_i - c_j.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, B, new, H, Hkv, d, page, length, **kw):
    c = dict(name=name, op=op, B=B, new=new, H=H, Hkv=Hkv, d=d, page=page, length=length, prefix=0, ragged=False,
             ragged_new=False, dtype="bf16", rotary="none", rot=0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token on a small model: nothing but latency
        _case("append_one_token", "append", 1, 1, 16, 16, 64, 64, 1000, rotary="half", rot=64),
        # a full serving batch's next tokens, grouped heads, keys rotated
        _case("append_batch_step", "append", 128, 1, 32, 8, 128, 64, 4096, ragged=True, rotary="half", rot=128),
        # prompts of several users entering the cache, ragged and odd lengths, half of each head rotated in pairs
        _case("append_prompts", "append", 6, 16384, 32, 8, 128, 64, 16384, ragged=True, ragged_new=True,
              rotary="pairs", rot=64),
        # a small fp32 model checked against its training code
        _case("append_prompt_f32", "append", 2, 257, 4, 4, 64, 16, 300, dtype="f32", rotary="half", rot=32),
        # one user, small model, a short odd context: latency
        _case("decode_short", "decode", 1, 1, 16, 16, 64, 64, 1000),
        # fp32, the framework's smallest parity shape and its ragged neighbours
        _case("decode_f32", "decode", 2, 1, 2, 2, 64, 16, 257, dtype="f32", ragged=True),
        # one user deep in a long context: the split over keys decides
        _case("decode_long_context", "decode", 1, 1, 32, 8, 128, 64, 65536),
        # a verification step of four guessed tokens, as many key heads as query heads
        _case("decode_guessed_tokens", "decode", 16, 4, 16, 16, 128, 32, 4096, ragged=True),
        # a full ragged serving batch: the cache's bandwidth decides
        _case("decode_batch", "decode", 64, 1, 32, 8, 128, 64, 16384, ragged=True),
        # a few continuations of one short odd prompt
        _case("shared_few", "shared", 4, 1, 16, 16, 64, 16, 33, prefix=777),
        # users of one assistant behind its long instructions
        _case("shared_instructions", "shared", 32, 1, 32, 8, 128, 64, 500, prefix=16384, ragged=True),
        # many questions about one long document
        _case("shared_document", "shared", 256, 1, 32, 8, 128, 64, 200, prefix=32768, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "shared"])
    H, Hkv = rng.choice([(16, 16), (32, 8), (32, 32), (12, 4), (14, 2), (8, 1), (16, 8)])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kw = dict(ragged=rng.random() < 0.7)
    if op == "append":
        if rng.random() < 0.5:
            B, new = _log_int(rng, 1, 128), rng.randint(1, 4)
            length = max(new, _log_int(rng, 8, 4096))
        else:
            B, new = _log_int(rng, 1, 6), _log_int(rng, 5, 8192)
            length = new + rng.randint(0, 500)
            kw["ragged_new"] = rng.random() < 0.5
        kw["rotary"] = rng.choice(["none", "half", "pairs"])
        kw["rot"] = 0 if kw["rotary"] == "none" else rng.choice([d, d // 2])
        kw["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        if kw["dtype"] == "f32":  # twice the bytes
            B = max(1, B // 2)
    elif op == "decode":
        B, new = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7])
        # at most the largest listed case's keys and values
        most = 64 * 16384 * 8 * 128 // (B * Hkv * d * max(1, new // 2))
        length = max(new, _log_int(rng, 16, max(32, min(65536, most))))
        if rng.random() < 0.15:
            kw["dtype"] = "f32"
            B, length = min(B, 4), max(new, min(length, 2048))
        kw["ragged_new"] = new > 1 and rng.random() < 0.5
    else:
        B, new = _log_int(rng, 2, 256), rng.choice([1, 1, 2])
        # at most the largest listed case's products, and 64 MB of fp32 scores a head
        most = min(256 * 32 * 32768 // (B * new * H), 16 * 1024 * 1024 * 4 // (B * new))
        kw["prefix"] = _log_int(rng, 100, max(200, min(32768, most)))
        length = max(new, _log_int(rng, 1, 512))
    return {k: v for k, v in _case("", op, B, new, H, Hkv, d, page, length, **kw).items() if k != "name"}


def _counts(case):
    """New tokens and own tokens (the new ones among them) of every sequence."""
    B, new, length = case["B"], case["new"], case["length"]
    n = [1 + (new - 1) * (B - b) // B if case["ragged_new"] else new for b in range(B)]
    # from the full length down to an eighth of it, in steps that are no multiple of a page
    own_len = [length - (b * 7919) % max(1, length * 7 // 8) if case["ragged"] else length for b in range(B)]
    return n, [max(x, y) for x, y in zip(own_len, n)]


def work(case):
    n, own_len = _counts(case)
    e = 2 if case["dtype"] == "bf16" else 4
    H, Hkv, d, rows = case["H"], case["Hkv"], case["d"], sum(n)
    if case["op"] == "append":
        turned = 2 * rows * H * d * e if case["rot"] else 0  # q in and out
        tables = rows * case["rot"] * 4
        return {"bytes": 4 * rows * Hkv * d * e + turned + tables + 2 * rows * H * 4, "flops": 0}
    keys = sum(own_len) + case["prefix"]
    seen = sum(x * (y + case["prefix"]) - x * (x - 1) // 2 for x, y in zip(n, own_len))  # (query, key) pairs a head
    return {"bytes": keys * (2 * Hkv * d * e + H * 4) + rows * H * (2 * d * e + 4), "flops": 4 * seen * H * d}


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


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    B, H, Hkv, d, S, P = (case[x] for x in ("B", "H", "Hkv", "d", "page", "prefix"))
    dt = _DTYPES[case["dtype"]]
    n, own_len = _counts(case)
    rows, nb, npre = sum(n), -(-max(own_len) // S), -(-P // S)

    def normal(*shape, dtype=dt):
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
    s = {
        "case": case,
        "k": normal(pages, Hkv, S, d),
        "v": normal(pages, Hkv, S, d),
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
    have = torch.tensor([y - x if case["op"] == "append" else y for x, y in zip(n, own_len)], device=dev)
    if int(have.max()) > 0:
        z = normal(B, nb * S, H, dtype=torch.float32) + head
        local, base = _gates(z, before, S)
        held = (col * S)[None] < have[:, None]
        within = (col[None, :, None] * S + torch.arange(S, device=dev)) < have[:, None, None]
        local = torch.where(within[:, :, None], local, 0.0)
        at = table.long()[held]
        s["g"][at], s["gbase"][at] = local[held], base[held]
        del z, local, base
    s["q"] = normal(rows, H, d)
    if case["op"] == "append":
        s["k_new"], s["v_new"] = normal(rows, Hkv, d), normal(rows, Hkv, d)
        s["z"] = normal(rows, H, dtype=torch.float32) + head
        s["cos"], s["sin"] = _tables(case, dev) if case["rot"] else (None, None)
    if own:  # the handles that a serving loop keeps: they hold the tensors above, and a workspace
        import forget_gated_softmax_gb300 as fox

        s["cache"] = fox.make_cache(s["k"], s["v"], s["g"], s["gbase"])
        s["batch"] = fox.make_batch(s["lens"], s["table"], cu_new=s["cu"], max_new=case["new"],
                                    prefix_table=s["prefix_table"], prefix_len=P)
        s["ws"] = fox.cache_workspace(s["cache"], s["batch"], rows)
    return s


def run(s):
    if own:
        import forget_gated_softmax_gb300 as fox

        case = s["case"]
        if case["op"] == "append":
            turned = fox.fox_cache_append(s["cache"], s["batch"], s["k_new"], s["v_new"], s["z"],
                                          q=s["q"] if case["rot"] else None, cos=s["cos"], sin=s["sin"],
                                          pairs=case["rotary"] == "pairs", ws=s["ws"])
            return s["k"], s["v"], s["g"], s["gbase"], turned
        return fox.fox_decode(s["cache"], s["batch"], s["q"], ws=s["ws"])
    return _append(s) if s["case"]["op"] == "append" else _attend(s)


# ------------------------------------------------------------------------------------- plain forms


def _rows(s):
    """Sequence and position of every new token."""
    B, rows = s["lens"].numel(), s["q"].shape[0]
    i = torch.arange(rows, device=s["q"].device)
    if s["cu"] is None:
        each = rows // B
        b = i // each
        return b, s["lens"][b].long() - each + i % each
    cu = s["cu"].long()
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, s["lens"][b].long() - (cu[b + 1] - i)


def _turn(x, cos, sin, pairs):
    """x [rows, heads, d] with its first 2 * cos.shape[1] channels rotated by the rows' angles."""
    x = x.float()
    r = cos.shape[1] * 2
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., : r // 2], x[..., r // 2 : r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _append(s):
    case, S = s["case"], s["case"]["page"]
    b, pos = _rows(s)
    page, slot = s["table"][b, pos // S].long(), pos % S
    k, q = s["k_new"], None
    if case["rot"]:
        cos, sin = s["cos"][pos], s["sin"][pos]
        k = _turn(k, cos, sin, case["rotary"] == "pairs").to(k.dtype)
        q = _turn(s["q"], cos, sin, case["rotary"] == "pairs").to(k.dtype)
    s["k"][page, :, slot] = k
    s["v"][page, :, slot] = s["v_new"]
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
    fresh = opens >= first
    o = torch.maximum(opens, first)
    base = torch.where(fresh[:, None], c[o] - a[o], s["gbase"][page].double().sum(-1))
    high = base.float()
    s["g"][page, :, slot] = (c - base).float()
    low = (base - high.double()).float()
    s["gbase"][page[fresh]] = torch.stack([high, low], -1)[fresh]
    return s["k"], s["v"], s["g"], s["gbase"], q


def _attend(s):
    case = s["case"]
    H, Hkv, d, S, P, B = (case[x] for x in ("H", "Hkv", "d", "page", "prefix", "B"))
    G = H // Hkv
    b, pos = _rows(s)
    t = pos - s["lens"][b].long() + case["new"]  # place in a padded [B, new] batch of rows
    dev = pos.device
    q = torch.zeros(B, case["new"], H, d, device=dev)
    q[b, t] = s["q"].float() / math.sqrt(d)
    q = q.view(B, -1, Hkv, G, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, new, d]
    table = s["table"].long()
    keys = torch.arange(table.shape[1] * S, device=dev)
    cum = s["gbase"][table].double().sum(-1)[..., None] + s["g"][table].double()  # [B, blocks, H, S]
    cum = cum.permute(0, 2, 1, 3).reshape(B, H, -1)
    at = (s["lens"].long()[:, None] - case["new"] + torch.arange(case["new"], device=dev) - P)  # own place of the rows
    ci = cum.gather(2, at.clamp(min=0)[:, None].expand(-1, H, -1))
    bias = (ci[..., None] - cum[:, :, None]).float()
    bias = torch.where(keys <= at[:, None, :, None], bias, -math.inf)  # [B, H, new, keys]
    k = s["k"][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, -1, d)
    score = (q @ k.transpose(-1, -2)).view(B, H, case["new"], -1) + bias
    del k, bias
    if P:
        pt = s["prefix_table"].long()
        kp = s["k"][pt].float().permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :P]
        vp = s["v"][pt].float().permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :P]
        cp = (s["gbase"][pt].double().sum(-1)[..., None] + s["g"][pt].double()).permute(1, 0, 2).reshape(H, -1)[:, :P]
        tall = q.permute(1, 2, 0, 3, 4).reshape(Hkv, -1, d)  # all rows of a key head against the one prefix
        sp = (tall @ kp.transpose(-1, -2)).view(H, B, case["new"], P)
        # c_i - c_j = (c_i - c_last) + (c_last - c_j), c_last the prefix's last token's
        sp = sp + (cp[:, -1:] - cp).float()[:, None, None] + (ci.permute(1, 0, 2) - cp[:, -1, None, None]).float()[..., None]
        most = torch.maximum(score.amax(-1), sp.amax(-1).permute(1, 0, 2))
        sp = torch.exp(sp - most.permute(1, 0, 2)[..., None])
    else:
        most = score.amax(-1)
    w = torch.exp(score - torch.where(torch.isfinite(most), most, 0.0)[..., None])
    total = w.sum(-1)
    v = s["v"][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, -1, d)
    v = torch.where((keys < (s["lens"].long() - P)[:, None])[:, None, None, :, None], v, 0.0)
    o = (w.view(B, Hkv, G, case["new"], -1) @ v).view(B, H, case["new"], d)
    if P:
        total = total + sp.sum(-1).permute(1, 0, 2)
        op = (sp.reshape(Hkv, -1, P) @ vp).view(H, B, case["new"], d)
        o = o + op.permute(1, 0, 2, 3)
    o, lse = o / total[..., None], most + torch.log(total)
    return o.permute(0, 2, 1, 3)[b, t].to(s["q"].dtype), lse.permute(0, 2, 1)[b, t].contiguous()


# ------------------------------------------------------------------------------------ exact values


def exact(case, seed):
    """The definition, one sequence after the other, in 64 bits."""
    s = prepare(case, seed)
    n, own_len = _counts(case)
    H, Hkv, d, S, P = (case[x] for x in ("H", "Hkv", "d", "page", "prefix"))
    dev = s["q"].device
    logf = lambda z: torch.nn.functional.logsigmoid(z.double())  # noqa: E731
    row = 0
    if case["op"] == "append":
        k, v, g, gb = (s[x].double() for x in ("k", "v", "g", "gbase"))
        turned = torch.empty(sum(n), H, d, dtype=torch.float64, device=dev) if case["rot"] else None
        for b, (new, length) in enumerate(zip(n, own_len)):
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
                turned[row : row + new] = qn
            k[page, :, slot], v[page, :, slot] = kn, s["v_new"][row : row + new].double()
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
        return k, v, g, gb, turned
    o = torch.empty(sum(n), H, d, dtype=torch.float64, device=dev)
    lse = torch.empty(sum(n), H, dtype=torch.float64, device=dev)
    for b, (new, length) in enumerate(zip(n, own_len)):
        ids = s["table"][b, : -(-length // S)].long()

        def flat(x, ids=ids, length=length):  # [pages, heads, S, ...] -> [heads, tokens, ...]
            y = x[ids].transpose(0, 1).flatten(1, 2)[:, :length].double()
            if P:
                y = torch.cat([x[s["prefix_table"].long()].transpose(0, 1).flatten(1, 2)[:, :P].double(), y], 1)
            return y

        key, val = flat(s["k"]), flat(s["v"])
        c = flat(s["gbase"].double().sum(-1)[..., None] + s["g"].double())
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
