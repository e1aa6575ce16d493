"""The serving operators over an 8-bit paged key/value cache: what is measured, and their plain forms.

A case is one pass through ``cache_append``, ``cache_attention`` or ``cache_evict`` (or the three as a decoding
step chains them).  Head counts and head dims are those of this repository's workloads (32/8 heads of 128, 8/8 of
64, 8 heads of 256); lengths run from one token to long contexts."""
import math

import torch

own = False

DEV = "cuda"
E4M3, I8 = torch.float8_e4m3fn, torch.int8
IO = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(name, op, **kw):
    base = dict(op=op, B=1, Hq=32, Hkv=8, D=128, page=64, kind="e4m3", io="bf16", L=1024, ragged=False, n=1)
    base.update(kw)
    if name:
        base["name"] = name
    return base


def listed():
    return [
        # one token of each of 32 running requests enters the cache: the smallest call, once per layer and step
        _case("append_step", "append", B=32, L=1990, ragged=True, n=1),
        # a whole prompt enters (the bench workload's batch, heads and length)
        _case("append_prompt", "append", B=2, L=0, n=4096),
        # pieces of prompts of unequal length continue half-filled pages, 8-bit integers
        _case("append_pieces_int8", "append", B=8, Hq=8, D=64, page=32, kind="int8", io="f16", L=2000, ragged=True,
              n=333),
        # one request decodes over a short context: latency
        _case("attn_one_short", "attn", B=1, L=1000),
        # a serving batch decodes, contexts of unequal length
        _case("attn_batch", "attn", B=32, L=8192, ragged=True),
        # one request decodes over a very long context
        _case("attn_one_long", "attn", B=1, L=131071),
        # no shared heads, small heads, 8-bit integers, short pages
        _case("attn_mha_int8", "attn", B=16, Hq=8, D=64, page=16, kind="int8", io="f16", L=4608),
        # four draft tokens are verified at once; heads of 256, softcap and a sliding window
        _case("attn_verify_d256", "attn", B=8, Hq=16, Hkv=8, D=256, page=128, L=6000, ragged=True, n=4, softcap=20.0,
              window=4096),
        # a piece of a long prompt attends to everything before it
        _case("attn_prompt_piece", "attn", B=2, L=16384, n=2048),
        # a decoding step that also accumulates the attention weight of every cached token
        _case("attn_tracked", "attn", B=16, L=4096, ragged=True, track=True),
        # prompts are cut down to their heaviest and latest tokens, into fresh pages
        _case("evict_prompt", "evict", B=8, L=16000, ragged=True, keep=2048, recent=64),
        # a decoding step under a fixed budget: append, attend with tracking, evict back to the budget in place
        _case("step_budget", "step", B=16, L=2048, n=1, keep=2048, recent=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "evict", "step"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = _case("", op, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 128, 256]),
              page=rng.choice([16, 32, 64, 128]), kind=rng.choice(["e4m3", "e4m3", "int8"]),
              io=rng.choice(["bf16", "f16"]), ragged=rng.random() < 0.6)
    if op == "append":
        c.update(B=_log(rng, 1, 64), n=_log(rng, 1, 1000), L=_log(rng, 1, 3000))
        if rng.random() < 0.3:
            c["io"] = "f32"
    elif op == "attn":
        c["n"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 700)])
        c["B"] = _log(rng, 1, 32 if c["n"] <= 8 else 6)
        room = 400_000_000 // (2 * Hkv * c["D"] * c["B"] * (1 + c["n"] // 128))
        c["L"] = c["n"] + _log(rng, 1, min(60000, max(600, room)))
        if rng.random() < 0.3:
            c["softcap"] = rng.choice([20.0, 50.0])
        if rng.random() < 0.3:
            c["window"] = _log(rng, 16, 4096)
        c["track"] = rng.random() < 0.3
    elif op == "evict":
        c.update(B=_log(rng, 1, 8), L=_log(rng, 300, 16000))
        c["keep"] = min(4000, max(8, int(c["L"] * rng.uniform(0.05, 0.6))))
        c["recent"] = int(c["keep"] * rng.uniform(0.0, 0.5))
    else:
        c.update(B=_log(rng, 1, 32), n=rng.randint(1, 4), ragged=False, L=_log(rng, 100, 4000))
        c["keep"], c["recent"] = c["L"], c["L"] // rng.randint(4, 16)
    return c


# ---------------------------------------------------------------- sizes that follow from a case


def _lens(c):
    """Tokens in the cache when the call starts (append, step) or in all (attn, evict), by sequence."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    least = c["n"] if c["op"] == "attn" else 1
    return [max(least, L - (L * 3 // 4) * ((i * 5) % 8) // 8) for i in range(B)]


def _news(c):
    """New tokens by sequence."""
    if c["ragged"] and c["op"] == "append":
        return [max(1, c["n"] - (c["n"] // 2) * (i % 3) // 2) for i in range(c["B"])]
    return [c["n"]] * c["B"]


def _visible(length, n, window):
    """(key, row) pairs that n rows at the end of `length` tokens see, and the tokens that any row sees."""
    pairs = 0
    for i in range(n):
        p = length - n + i + 1
        pairs += min(p, window) if window else p
    return pairs, min(length, window + n - 1) if window else length


def work(case):
    c, esz = case, 4 if case["io"] == "f32" else 2
    tok = 2 * c["Hkv"] * c["D"]  # bytes and elements of one cached token
    q = c["B"] * c["Hq"] * c["n"] * (2 * c["D"] * esz + 4)
    seen = [_visible(x + (c["n"] if c["op"] == "step" else 0), c["n"], c.get("window", 0)) for x in _lens(c)]
    flops = 4 * c["Hq"] * c["D"] * sum(p for p, _ in seen)
    read = sum(t for _, t in seen) * tok
    tracked = sum(t for _, t in seen) * c["Hkv"] * 8
    new = sum(_news(c)) * tok * (esz + 1)
    if c["op"] == "append":
        return {"bytes": new, "flops": 2 * sum(_news(c)) * tok}
    if c["op"] == "attn":
        return {"bytes": read + q + (tracked if c.get("track") else 0), "flops": flops}
    if c["op"] == "evict":
        kept = sum(min(x, c["keep"]) for x in _lens(c))
        return {"bytes": sum(_lens(c)) * c["Hkv"] * 8 + kept * (2 * tok + 8 * c["Hkv"]), "flops": sum(_lens(c)) * c["Hkv"]}
    moved = c["B"] * c["n"] * 2 * tok
    return {"bytes": new + read + q + tracked + sum(x + c["n"] for x in _lens(c)) * c["Hkv"] * 8 + moved, "flops": flops}


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 % (1 << 62) + 17)
    B, H, D, page, op = c["B"], c["Hkv"], c["D"], c["page"], c["op"]
    lens, news = _lens(c), _news(c)
    total = [a + (b if op in ("append", "step") else 0) for a, b in zip(lens, news)]
    need = [max(1, -(-t // page)) for t in total]
    dst = [-(-c["keep"] // page)] * B if op == "evict" else [0] * B
    M, P = max(need), sum(need) + sum(dst) + 3
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32).tolist()

    def table(counts, width):  # pages in no order; entries that no token needs are -1
        rows = []
        for k in counts:
            rows.append([order.pop() for _ in range(k)] + [-1] * (width - k))
        return torch.tensor(rows, dtype=torch.int32, device=DEV)

    randn = lambda *s, **k: torch.randn(*s, generator=g, device=DEV, **k)  # noqa: E731
    kind = E4M3 if c["kind"] == "e4m3" else I8
    spread, top = (100.0, 448.0) if kind == E4M3 else (40.0, 127.0)

    def pool():
        x = torch.empty(P, H, page, D, dtype=kind, device=DEV)
        step = max(1, (1 << 26) // (H * page * D))
        for i in range(0, P, step):
            y = randn(min(step, P - i), H, page, D).mul_(spread).clamp_(-top, top)
            x[i:i + step] = (y.round_() if kind == I8 else y).to(kind)
        s = torch.randint(-7, -4, (P, H), generator=g, device=DEV).float().exp2_()
        return x, s * (2.0 if kind == I8 else 1.0)

    s = dict(case=dict(c), table=table(need, M), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    s["k"], s["ks"] = pool()
    s["v"], s["vs"] = pool()
    n, io = c["n"], IO[c["io"]]
    if op in ("append", "step"):
        s["new_k"], s["new_v"] = (randn(B, H, n, D).to(io) for _ in range(2))
        s["news"] = torch.tensor(news, dtype=torch.int32, device=DEV)
    if op in ("attn", "step"):
        s["q"] = randn(B, c["Hq"], n, D).to(io)
    W = M * page
    if op in ("evict", "step") or c.get("track"):
        # a few tokens carry most of the weight, as in a trained model
        s["weights"] = randn(B, H, W).mul_(2.0).exp_()
    if op in ("evict", "step"):
        s["positions"] = torch.arange(W, dtype=torch.int32, device=DEV).expand(B, H, W).contiguous()
    if op == "step":
        s["seen"] = s["lens"].clone()
    if op == "evict":
        s["into"] = table(dst, max(dst))
        s["weights_out"] = torch.zeros(B, H, c["keep"], device=DEV)
        s["positions_out"] = torch.zeros(B, H, c["keep"], dtype=torch.int32, device=DEV)
    if own:
        import attention_forward_08_gb300 as fa
        s["cache"] = fa.KVCache(s["k"], s["v"], s["ks"], s["vs"])
    return s


# ---------------------------------------------------------------- plain forms


def _top(kind):  # the largest value as (mantissa in [0.5, 1), exponent, value)
    return (0.875, 9, 448.0) if kind == E4M3 else (0.9921875, 7, 127.0)


def _pow2_scale(amax, kind):
    """The least power of two s with amax <= MAX * s, at least 2^-100."""
    m0, e0, _ = _top(kind)
    m, e = torch.frexp(amax)
    e = e - e0 + (m > m0).to(e.dtype)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -100).clamp_min(-100))


def _round8(x, kind):
    top = _top(kind)[2]
    x = x.clamp(-top, top)
    return x.to(E4M3) if kind == E4M3 else torch.nan_to_num(x, nan=0.0).round().to(I8)


def _bytes(pool):  # indexing on the stored bytes works for both kinds
    return pool.view(torch.uint8)


def _append_one(pool, scale, x, table, lens, news):
    kind, page = pool.dtype, pool.shape[2]
    P, H, _, D = pool.shape
    n = x.shape[2]
    x = x.float()
    b, t = torch.nonzero(torch.arange(n, device=x.device) < news[:, None], as_tuple=True)
    pos = lens.long()[b] + t
    at, slot = table[b, pos // page].long(), pos % page
    x = x.transpose(1, 2)[b, t]  # [tokens, H, D]
    a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
    first = torch.full((P,), page, dtype=torch.long, device=x.device).scatter_reduce(0, at, slot, "amin")
    amax = torch.zeros(P, H, device=x.device).scatter_reduce(0, at[:, None].expand(-1, H), a, "amax")
    touched, held = first < page, (first > 0) & (first < page)
    old = torch.where(held[:, None], scale, 0.0)
    new = torch.where(touched[:, None], torch.maximum(old, _pow2_scale(amax, kind)), scale)
    grown = torch.nonzero(held[:, None] & (new > scale), as_tuple=True)
    blocks = pool[grown].float() * (scale[grown] / new[grown])[:, None, None]
    live = torch.arange(page, device=x.device) < first[grown[0]][:, None]
    _bytes(pool)[grown] = torch.where(live[..., None], _bytes(_round8(blocks, kind)), _bytes(pool)[grown])
    _bytes(pool)[at, :, slot] = _bytes(_round8(x / new[at][..., None], kind))
    scale.copy_(new)


def _plain_append(s):
    _append_one(s["k"], s["ks"], s["new_k"], s["table"], s["lens"], s["news"])
    _append_one(s["v"], s["vs"], s["new_v"], s["table"], s["lens"], s["news"])


def _tokens(pool, scale, table):
    """[B, H, M * page, D] in fp32."""
    at = table.long().clamp_min(0)
    x = pool[at].float() * scale[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(s, lens):
    c, q = s["case"], s["q"]
    B, Hq, n, D = q.shape
    H, W = c["Hkv"], s["table"].shape[1] * c["page"]
    k, v = _tokens(s["k"], s["ks"], s["table"]), _tokens(s["v"], s["vs"], s["table"])
    x = torch.matmul(q.float().reshape(B, H, -1, D), k.transpose(2, 3)) / math.sqrt(D)
    if c.get("softcap"):
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.view(B, H, Hq // H, n, W)
    j = torch.arange(W, device=q.device)
    pos = (lens.long()[:, None] - n + torch.arange(n, device=q.device))[..., None]
    see = j <= pos
    if c.get("window"):
        see = see & (j > pos - c["window"])
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e38)
    p = torch.exp(x - m)
    del x
    l = p.sum(-1, keepdim=True)
    p = p / l.clamp_min(1e-38)
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, H, -1, W), v).view(B, Hq, n, D).to(q.dtype)
    lse = (m + torch.log(l)).view(B, Hq, n)
    if "weights" in s:
        s["weights"] += p.sum((2, 3))
    return o, lse


def _plain_evict(s, lens, into):
    c, w, pos = s["case"], s["weights"], s["positions"]
    keep, page, table = c["keep"], c["page"], s["table"]
    B, H, W = w.shape
    j = torch.arange(W, device=w.device)
    n = lens.long()[:, None, None]
    held = (j < n).expand(B, H, W)
    late = pos > torch.where(held, pos, -1).amax(2, keepdim=True) - c["recent"]
    rank = torch.where(late, math.inf, torch.nan_to_num(w, nan=-math.inf, posinf=math.inf, neginf=-math.inf))
    rank = torch.where(held, rank, -math.inf)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    count = n.clamp_max(keep)  # [B, 1, 1]
    kept = torch.zeros_like(held).scatter(2, order, (j < count).expand(B, H, W))
    slots = j[:keep]
    if into is None:  # kept slots past the budget go to the free ones below it
        from_ = torch.sort((kept & (j >= keep)).to(torch.int8), dim=2, descending=True, stable=True).indices[..., :keep]
        hole = ~kept[..., :keep] & (slots < count)
        nth = (hole.cumsum(2) - 1).clamp_min(0)
        src = torch.where(hole, from_.gather(2, nth), slots)
    else:
        src = torch.sort(kept.to(torch.int8), dim=2, descending=True, stable=True).indices[..., :keep]
    live = (slots < count).expand(B, H, keep)
    src = torch.where(live, src, 0)
    to = table if into is None else into
    b, h, d = torch.nonzero(live & ((src != slots) if into is None else live), as_tuple=True)
    at = src[b, h, d]
    # the scale of a block is the largest of its tokens' blocks
    pages_of = lambda t, x: t.long()[torch.arange(B, device=w.device)[:, None, None], x // page]  # noqa: E731
    head = torch.arange(H, device=w.device)[None, :, None]
    blocks = -(-keep // page)
    for pool, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        kind = pool.dtype
        theirs = torch.where(live, scale[pages_of(table, src), head], 0.0)
        theirs_by_block = torch.nn.functional.pad(theirs, (0, blocks * page - keep)).view(B, H, blocks, page)
        used = to.long()[:, :blocks][:, None].expand(B, H, blocks)
        at_all = pages_of(to, slots.expand(B, H, keep))
        new = theirs_by_block.amax(3)
        x = pool[pages_of(table, src)[b, h, d], h, at % page].float()
        mine = new[b, h, d // page]
        x = x * (theirs[b, h, d] / mine)[:, None]
        if into is None:  # tokens that stay in a block whose scale grows
            old = scale[used.clamp_min(0), head]
            gb, gh, gd = torch.nonzero(live & (src == slots) & (new > old).repeat_interleave(page, 2)[..., :keep],
                                       as_tuple=True)
            stay = pool[at_all[gb, gh, gd], gh, gd % page].float()
            stay = stay * (old[gb, gh, gd // page] / new[gb, gh, gd // page])[:, None]
            _bytes(pool)[at_all[gb, gh, gd], gh, gd % page] = _bytes(_round8(stay, kind))
        _bytes(pool)[at_all[b, h, d], h, d % page] = _bytes(_round8(x, kind))
        some = live[..., ::page]
        i = torch.nonzero(some, as_tuple=True)
        scale[used[i], i[1]] = new[i]
    w_out, p_out = (w, pos) if into is None else (s["weights_out"], s["positions_out"])
    new_w, new_p = w.gather(2, src), pos.gather(2, src)
    w_out[..., :keep] = torch.where(live, new_w, w_out[..., :keep])
    p_out[..., :keep] = torch.where(live, new_p, p_out[..., :keep])
    return lens.clamp_max(keep)


def _plain_track_new(s):
    """New slots start without weight, at the positions that follow those seen."""
    t = torch.arange(s["case"]["n"], device=DEV)
    at = (s["lens"].long()[:, None] + t)[:, None].expand(-1, s["case"]["Hkv"], -1)
    s["weights"].scatter_(2, at, 0.0)
    s["positions"].scatter_(2, at, (s["seen"][:, None] + t).to(torch.int32)[:, None].expand_as(at))


def run(state):
    s, c = state, state["case"]
    op, opt = c["op"], {k: c[k] for k in ("softcap", "window") if k in c}
    if own:
        import attention_forward_08_gb300 as fa
        if op == "append":
            fa.cache_append(s["cache"], s["new_k"], s["new_v"], s["table"], s["lens"], n_new=s["news"])
        elif op == "attn":
            o, lse = fa.cache_attention(s["q"], s["cache"], s["table"], s["lens"], weights=s.get("weights"), **opt)
        elif op == "evict":
            lens = fa.cache_evict(s["cache"], s["table"], s["lens"], s["weights"], s["positions"], keep=c["keep"],
                                  recent=c["recent"], into=s["into"], weights_out=s["weights_out"],
                                  positions_out=s["positions_out"])
        else:
            fa.cache_append(s["cache"], s["new_k"], s["new_v"], s["table"], s["lens"], weights=s["weights"],
                            positions=s["positions"], seen=s["seen"])
            o, lse = fa.cache_attention(s["q"], s["cache"], s["table"], s["lens"] + c["n"], weights=s["weights"])
            lens = fa.cache_evict(s["cache"], s["table"], s["lens"] + c["n"], s["weights"], s["positions"],
                                  keep=c["keep"], recent=c["recent"])
            s["seen"] += c["n"]
    elif op == "append":
        _plain_append(s)
    elif op == "attn":
        o, lse = _plain_attention(s, s["lens"])
    elif op == "evict":
        lens = _plain_evict(s, s["lens"], s["into"])
    else:
        _plain_append(s)
        _plain_track_new(s)
        o, lse = _plain_attention(s, s["lens"] + c["n"])
        lens = _plain_evict(s, s["lens"] + c["n"], None)
        s["seen"] += c["n"]
    pools = dict(k=s["k"], v=s["v"], k_scale=s["ks"], v_scale=s["vs"])
    if op == "append":
        return pools
    if op == "attn":
        return dict(o=o, lse=lse, **({"weights": s["weights"]} if c.get("track") else {}))
    if op == "evict":
        return dict(pools, lens=lens, weights=s["weights_out"], positions=s["positions_out"])
    return dict(pools, o=o, lse=lse, lens=lens, weights=s["weights"], positions=s["positions"])


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_attention(s, lens):
    """Sequence by sequence, over the tokens that it holds."""
    c, q = s["case"], s["q"]
    B, Hq, n, D = q.shape
    H, page = c["Hkv"], c["page"]
    cap, window = c.get("softcap", 0.0), c.get("window", 0)
    o, lse = torch.zeros(B, Hq, n, D, dtype=torch.float64, device=DEV), torch.empty(B, Hq, n, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if "weights" in s else None
    for b in range(B):
        L = int(lens[b])
        pages = s["table"][b, :-(-L // page)].long()
        take = lambda x, y: (x[pages].double() * y[pages].double()[:, :, None, None]).transpose(0, 1).reshape(H, -1, D)[:, :L]  # noqa: E731
        k, v = take(s["k"], s["ks"]), take(s["v"], s["vs"])
        i = torch.arange(L - n, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None]
        hidden = (j > i) | ((j <= i - window) if window else (j < 0))
        for h in range(H):
            rows = slice(h * (Hq // H), (h + 1) * (Hq // H))
            z = torch.einsum("gid,jd->gij", q[b, rows].double(), k[h]) * D ** -0.5
            if cap:
                z = torch.tanh(z / cap) * cap
            z[:, hidden] = -math.inf
            y = torch.logsumexp(z, -1)
            z = torch.exp(z - y[..., None])
            lse[b, rows] = y
            o[b, rows] = torch.einsum("gij,jd->gid", z, v[h])
            if weights is not None:
                weights[b, h, :L] += z.sum((0, 1))
    return o, lse, weights


def _exact_round(x, kind):
    """To the nearest value of the type, ties to even, on its grid."""
    top = _top(kind)[2]
    x = x.clamp(-top, top)
    if kind == I8:
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    """Block by block of every sequence."""
    got = {}
    for name, new in (("k", s["new_k"]), ("v", s["new_v"])):
        kind, page = s[name].dtype, s[name].shape[2]
        pool, scale = s[name].double(), s[name + "s"].double()
        for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["news"].tolist())):
            for m in range(L // page, (L + n - 1) // page + 1):
                lo, hi = max(L, m * page), min(L + n, (m + 1) * page)
                at, old = int(s["table"][b, m]), lo - m * page
                x = new[b, :, lo - L:hi - L].double()
                e = torch.ceil(torch.log2(x.abs().amax((1, 2)) / _top(kind)[2])).clamp_min(-100)
                t = torch.exp2(e)
                if old:
                    t = torch.maximum(t, scale[at])
                    pool[at, :, :old] = _exact_round(pool[at, :, :old] * (scale[at] / t)[:, None, None], kind)
                pool[at, :, old:old + hi - lo] = _exact_round(x / t[:, None, None], kind)
                scale[at] = t
        got[name], got[name + "_scale"] = pool if kind == E4M3 else None, scale
    return got


def exact(case, seed):
    if case["op"] == "evict":  # copies, counts: nothing that either side approximates
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attn":
        o, lse, w = _exact_attention(s, s["lens"])
        return dict(o=o, lse=lse, **({"weights": w} if case.get("track") else {}))
    _plain_append(s)  # whole pools of stored values: the attention reads what was written
    _plain_track_new(s)
    o, lse, _ = _exact_attention(s, s["lens"] + case["n"])
    return dict(k=None, v=None, k_scale=None, v_scale=None, o=o, lse=lse, lens=None, weights=None, positions=None)
