"""Decoding with drafted tokens over an 8-bit paged cache: what is measured, and the operators' plain forms.

A case is one pass through ``cache_attention`` with a tree of drafts, through ``verify_drafts`` or ``cache_accept``, or
through a whole step (append, attend, verify, accept).  Head counts and head dims are those of this repository's
workloads (32/8 heads of 128, 8/8 of 64, 16/8 of 256); trees hold from one draft to two hundred, vocabularies from a
thousand tokens to 131072."""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3, I8 = torch.float8_e4m3fn, torch.int8
IO = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(name, op, **kw):
    base = dict(op=op, B=1, Hq=32, Hkv=8, D=128, page=64, kind="e4m3", io="bf16", L=1000, ragged=False, n=8,
                tree="beam", V=32000, drafts="sampled")
    base.update(kw)
    if name:
        base["name"] = name
    return base


def listed():
    return [
        # one request, eight drafts over a short context: the smallest call, latency
        _case("tree_one_small", "attn", B=1, n=8, L=1000),
        # a serving batch, sixteen drafts each over contexts of unequal length
        _case("tree_batch", "attn", B=16, n=16, L=8192, ragged=True),
        # many drafts a request
        _case("tree_wide", "attn", B=8, n=60, L=6000, ragged=True, tree="wide"),
        # no shared heads, small heads, 8-bit integers, short pages, one tree for all requests
        _case("tree_mha_int8", "attn", B=16, Hq=8, D=64, page=16, kind="int8", io="f16", L=4608, n=33, shared=True),
        # heads of 256, softcap and a sliding window
        _case("tree_d256", "attn", B=8, Hq=16, D=256, page=128, L=6000, ragged=True, n=13, softcap=20.0, window=4096),
        # one request over a very long context
        _case("tree_one_long", "attn", B=1, n=26, L=131071),
        # one request's chain of four drafts is verified: the smallest call
        _case("verify_one", "verify", B=1, n=5, tree="chain", V=32000),
        # a batch's trees, sampled from the draft model, an odd vocabulary
        _case("verify_batch", "verify", B=32, n=16, V=128001),
        # a batch's trees of most likely tokens (no draft probabilities), 16-bit probabilities cut to the likely tokens
        _case("verify_candidates", "verify", B=64, n=60, V=100000, drafts="likely", io="bf16", cut=True),
        # accepted drafts of a batch are brought together in the cache of one layer
        _case("accept_batch", "accept", B=32, n=16, L=2000, ragged=True),
        # long paths, 8-bit integers, wide heads, short pages
        _case("accept_long_int8", "accept", B=64, Hq=8, D=256, page=16, kind="int8", L=600, ragged=True, n=200),
        # a whole step of one layer: append the drafts, attend (tracking weights), verify, accept
        _case("step", "step", B=16, n=16, L=4096, track=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "verify", "verify", "accept", "step"])
    Hkv = rng.choice([1, 2, 4, 8])
    c = _case("", op, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 128, 256]),
              page=rng.choice([16, 32, 64, 128]), kind=rng.choice(["e4m3", "e4m3", "int8"]),
              io=rng.choice(["bf16", "f16"]), ragged=rng.random() < 0.6, tree=rng.choice(["beam", "beam", "wide", "chain"]))
    if op == "attn":
        c["n"] = _log(rng, 1, 200)
        c["B"] = _log(rng, 1, 32 if c["n"] <= 32 else 8)
        room = 300_000_000 // (2 * Hkv * c["D"] * c["B"] * (1 + c["n"] * c["Hq"] // Hkv // 256))
        c["L"] = c["n"] + _log(rng, 1, min(60000, max(600, room)))
        c["shared"] = rng.random() < 0.3
        if rng.random() < 0.3:
            c["softcap"] = rng.choice([20.0, 50.0])
        if rng.random() < 0.3:
            c["window"] = _log(rng, 16, 4096)
        c["track"] = rng.random() < 0.25
    elif op == "verify":
        c["n"], c["V"] = _log(rng, 2, 64), _log(rng, 1000, 131072)
        c["B"] = _log(rng, 1, max(2, min(64, 70_000_000 // (c["n"] * c["V"]))))
        c["io"] = rng.choice(["f32", "f32", "bf16", "f16"])
        c["drafts"], c["cut"] = rng.choice(["sampled", "sampled", "likely"]), rng.random() < 0.3
    elif op == "accept":
        c["n"] = _log(rng, 2, 200)
        c.update(B=_log(rng, 1, 64), L=c["n"] + _log(rng, 1, 600))
        c["track"] = rng.random() < 0.5
    else:
        c["n"] = _log(rng, 2, 32)
        c.update(B=_log(rng, 1, 16), L=c["n"] + _log(rng, 1, 4000), V=_log(rng, 1000, 32000), track=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- sizes that follow from a case


def _lens(c):
    """Tokens in the cache, the drafts among them."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    return [max(c["n"], L - (L * 3 // 4) * ((i * 5) % 8) // 8) for i in range(B)]


def work(case):
    c, n = case, case["n"]
    esz = 4 if c["io"] == "f32" else 2
    tok = 2 * c["Hkv"] * c["D"]  # bytes of one cached token
    lens = _lens(c)
    seen = [min(x, c["window"] + n) if c.get("window") else x for x in lens]
    attn = dict(bytes=sum(seen) * tok + c["B"] * c["Hq"] * n * (4 * c["D"] + 4) +
                (sum(seen) * c["Hkv"] * 8 if c.get("track") else 0),
                flops=4 * c["Hq"] * c["D"] * sum((x - n + 1) * n for x in seen))
    rows = 1 if c["drafts"] == "likely" else 2  # of the vocabulary's length, for the node where the path ends
    verify = dict(bytes=c["B"] * (rows * c["V"] * (4 if c["op"] == "step" else esz) + 16 * n),
                  flops=c["B"] * c["V"] * (3 if rows == 2 else 1))
    if c["op"] == "attn":
        return attn
    if c["op"] == "verify":
        return verify
    moved = c["B"] * sum(_depths(c["n"])) // len(_depths(c["n"]))  # tokens of an accepted path, on average
    accept = dict(bytes=2 * moved * tok, flops=moved * tok)
    if c["op"] == "accept":
        return accept
    new = c["B"] * n * tok * 3  # 16-bit values in, 8-bit values out
    return dict(bytes=new + attn["bytes"] + verify["bytes"] + accept["bytes"], flops=attn["flops"] + verify["flops"])


def _depths(n):
    """Lengths that an accepted path of n drafts is given."""
    return [1 + (n - 1) * k // 16 for k in range(1, 6)]


# ---------------------------------------------------------------- inputs


def _parents(c, rng):
    """A tree of n drafts: node 0 is the last token, whose own keys are not in the cache yet."""
    n = c["n"]
    if c["tree"] == "chain":
        return [i - 1 for i in range(n)]
    if c["tree"] == "wide":
        return [-1] + [rng.randrange(i) for i in range(1, n)]
    rows, level, wide = [-1], [0], 2 + n // 16  # levels of equal width, siblings side by side
    while len(rows) < n:
        picks = sorted(rng.choice(level) for _ in range(min(wide, n - len(rows))))
        level = list(range(len(rows), len(rows) + len(picks)))
        rows += picks
    return rows


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 % (1 << 62) + 29)
    rng = random.Random(int(seed) * 7 + 5)
    B, H, D, page, op, n = c["B"], c["Hkv"], c["D"], c["page"], c["op"], c["n"]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    trees = [_parents(c, rng) for _ in range(1 if c.get("shared") else B)]
    s = dict(case=dict(c), tree=i32(trees[0] if c.get("shared") else trees))
    if op != "verify":
        lens = _lens(c)
        need = [max(1, -(-t // page)) for t in lens]
        M, P = max(need), sum(need) + 3
        order = torch.randperm(P, generator=g, device=DEV).to(torch.int32).tolist()
        # pages in no order; entries that no token needs are -1
        s["table"] = i32([[order.pop() for _ in range(k)] + [-1] * (M - k) for k in need])
        s["lens"] = i32(lens)
        kind = E4M3 if c["kind"] == "e4m3" else I8
        spread, top = (100.0, 448.0) if kind == E4M3 else (40.0, 127.0)

        def pool():
            x = torch.empty(P, H, page, D, dtype=kind, device=DEV)
            step = max(1, (1 << 26) // (H * page * D))
            for i in range(0, P, step):
                y = randn(min(step, P - i), H, page, D).mul_(spread).clamp_(-top, top)
                x[i:i + step] = (y.round_() if kind == I8 else y).to(kind)
            e = torch.randint(-7, -4, (P, H), generator=g, device=DEV).float().exp2_()
            return x, e * (2.0 if kind == I8 else 1.0)

        s["k"], s["ks"] = pool()
        s["v"], s["vs"] = pool()
        if c.get("track"):  # a few tokens carry most of the weight, as in a trained model
            s["weights"] = randn(B, H, M * page).mul_(2.0).exp_()
        if own:
            import attention_forward_08_gb300 as fa
            s["cache"] = fa.KVCache(s["k"], s["v"], s["ks"], s["vs"])
    if op in ("attn", "step"):
        s["q"] = randn(B, c["Hq"], n, D).to(IO[c["io"]])
    if op == "step":
        s["new_k"], s["new_v"] = (randn(B, H, n, D).to(IO[c["io"]]) for _ in range(2))
        s["before"] = s["lens"] - n
    if op in ("verify", "step"):
        io = torch.float32 if op == "step" else IO[c["io"]]
        V, parent = c["V"], s["tree"].long().clamp_min(0)
        s["p"] = torch.empty(B, n, V, dtype=io, device=DEV)
        tokens = torch.zeros(B, n, dtype=torch.int32, device=DEV)
        if c["drafts"] == "sampled":
            s["p_draft"] = torch.empty(B, n, V, dtype=io, device=DEV)
        # a node's place among its siblings: likely candidates are distinct
        rank = (torch.tril(parent[:, :, None] == parent[:, None, :], -1).sum(2) - (parent == 0).int()).clamp_min(0)
        for b in range(B):  # (logits of one request at a time: they would not all fit beside the probabilities)
            z = randn(n, V).mul_(4.0)
            q = torch.softmax(z, -1)
            p = torch.softmax(z.add_(randn(n, V).mul_(0.8)), -1)
            if c.get("cut"):  # unlikely tokens are never sampled
                p = torch.where(p >= 0.02 * p.amax(-1, keepdim=True), p, 0.0)
                p /= p.sum(-1, keepdim=True)
            s["p"][b] = p.to(io)
            if c["drafts"] == "sampled":
                s["p_draft"][b] = q.to(io)
                tokens[b] = torch.multinomial(q[parent[b]], 1, generator=g)[:, 0].to(torch.int32)
            else:
                best = torch.topk(q, min(n, V), dim=-1).indices
                tokens[b] = best[parent[b], rank[b]].to(torch.int32)
        s["tokens"] = tokens
        s["u"] = torch.rand(B, n, generator=g, device=DEV)
        s["u_next"] = torch.rand(B, generator=g, device=DEV)
    if op == "accept":
        path = torch.full((B, n), -1, dtype=torch.int32)
        count = [rng.choice(_depths(n)) for _ in range(B)]
        for b in range(B):
            path[b, :count[b]] = torch.tensor([0] + sorted(rng.sample(range(1, n), count[b] - 1)), dtype=torch.int32)
        s["path"], s["count"] = path.to(DEV), i32(count)
    return s


# ---------------------------------------------------------------- plain forms


def _top(kind):  # the largest value as (mantissa in [0.5, 1), exponent, value)
    return (0.875, 9, 448.0) if kind == E4M3 else (0.9921875, 7, 127.0)


def _round8(x, kind):
    top = _top(kind)[2]
    x = x.clamp(-top, top)
    return x.to(E4M3) if kind == E4M3 else torch.nan_to_num(x, nan=0.0).round().to(I8)


def _bytes(pool):  # indexing on the stored bytes works for both kinds
    return pool.view(torch.uint8)


def _plain_append(pool, scale, x, table, lens):
    """n new tokens behind `lens`; a block's scale is the least power of two that they fit under, or its own."""
    kind, page = pool.dtype, pool.shape[2]
    P, H, _, D = pool.shape
    B, _, n, _ = x.shape
    x = x.float().transpose(1, 2).reshape(B * n, H, D)
    b = torch.arange(B, device=x.device).repeat_interleave(n)
    pos = (lens.long()[:, None] + torch.arange(n, device=x.device)).flatten()
    at, slot = table[b, pos // page].long(), pos % page
    first = torch.full((P,), page, dtype=torch.long, device=x.device).scatter_reduce(0, at, slot, "amin")
    amax = torch.zeros(P, H, device=x.device).scatter_reduce(0, at[:, None].expand(-1, H), x.abs().amax(2), "amax")
    m0, e0, _ = _top(kind)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - e0 + (m > m0).to(e.dtype), -100).clamp_min(-100)
    touched, held = first < page, (first > 0) & (first < page)
    old = torch.where(held[:, None], scale, 0.0)
    new = torch.where(touched[:, None], torch.maximum(old, torch.ldexp(torch.ones_like(amax), e)), scale)
    grown = torch.nonzero(held[:, None] & (new > scale), as_tuple=True)
    blocks = pool[grown].float() * (scale[grown] / new[grown])[:, None, None]
    live = torch.arange(page, device=x.device) < first[grown[0]][:, None]
    _bytes(pool)[grown] = torch.where(live[..., None], _bytes(_round8(blocks, kind)), _bytes(pool)[grown])
    _bytes(pool)[at, :, slot] = _bytes(_round8(x / new[at][..., None], kind))
    scale.copy_(new)


def _ancestors(tree):
    """[B, n, n]: does node i have node j above it, or is it j; and its depth."""
    n = tree.shape[1]
    up = (tree[..., None] == torch.arange(n, device=tree.device)).float()
    reach = up + torch.eye(n, device=tree.device)
    for _ in range(max(1, (n - 1).bit_length())):  # ways of twice the length each time
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0, reach.sum(2).long() - 1


def _tokens(pool, scale, table):
    """[B, H, M * page, D] in fp32."""
    at = table.long().clamp_min(0)
    x = pool[at].float() * scale[at][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    c, q, lens = s["case"], s["q"], s["lens"].long()
    B, Hq, n, D = q.shape
    H, W = c["Hkv"], s["table"].shape[1] * c["page"]
    k, v = _tokens(s["k"], s["ks"], s["table"]), _tokens(s["v"], s["vs"], s["table"])
    x = torch.matmul(q.float().reshape(B, H, -1, D), k.transpose(2, 3)) / math.sqrt(D)
    if c.get("softcap"):
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.view(B, H, Hq // H, n, W)
    above, depth = _ancestors(s["tree"].expand(B, n))
    j = torch.arange(W, device=q.device)
    base = (lens - n)[:, None, None]
    node = (j - base).clamp(0, n - 1).expand(B, n, W)  # the draft in slot j, if it is one
    see = torch.where(j < base, True, (j < lens[:, None, None]) & above.gather(2, node))
    if c.get("window"):
        at = torch.where(j < base, j, base + depth[:, None, :].expand(B, n, n).gather(2, node))
        see = see & (at > base + depth[..., None] - c["window"])
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e38)
    p = torch.exp(x - m)
    del x
    l = p.sum(-1, keepdim=True)
    p = p / l
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, H, -1, W), v).view(B, Hq, n, D).to(q.dtype)
    lse = (m + torch.log(l)).view(B, Hq, n)
    if "weights" in s:
        s["weights"] += p.sum((2, 3))
    return o, lse


def _plain_verify(s):
    """Nodes in order; a node is tested if its parent is where the path ends so far."""
    p, tree, tokens, u = s["p"], s["tree"].long(), s["tokens"].long(), s["u"].double()
    q = s.get("p_draft")
    B, n, V = p.shape
    b = torch.arange(B, device=p.device)
    cur = torch.zeros(B, dtype=torch.long, device=p.device)
    count = torch.ones_like(cur)
    path = torch.full((B, n + 1), -1, dtype=torch.int32, device=p.device)
    path[:, 0] = 0
    left = p[:, 0].double()  # what is left of the target's probabilities at the path's end
    taken = torch.zeros(B, dtype=torch.float64, device=p.device)
    z = torch.ones_like(taken)
    for i in range(1, n):
        t, test = tokens[:, i], tree[:, i] == cur
        r = left[b, t]
        draft = z if q is None else z * q[b, cur, t].double()
        yes = test & (u[:, i] * draft < r)
        no = test & ~yes
        if q is None:
            z = torch.where(no, z - r, z)
            left = left.scatter(1, t[:, None], torch.where(no, 0.0, r)[:, None])
        else:
            taken = torch.where(no, taken + z, taken)
            less = (p[b, cur].double() - taken[:, None] * q[b, cur].double()).clamp_min(0.0)
            left = torch.where(no[:, None], less, left)
            z = torch.where(no, left.sum(1), z)
        cur = torch.where(yes, i, cur)
        left = torch.where(yes[:, None], p[b, cur].double(), left)
        z, taken = torch.where(yes, 1.0, z), torch.where(yes, 0.0, taken)
        path.scatter_(1, torch.where(yes, count, n)[:, None], torch.full_like(path[:, :1], i))
        count = count + yes.long()
    path = torch.where(torch.arange(n, device=p.device) < count[:, None], path[:, :n], -1)
    left = torch.where((left.sum(1) > 0)[:, None], left, p[b, cur].double())
    sums = left.cumsum(1)
    token = (sums <= (s["u_next"].double() * sums[:, -1])[:, None]).sum(1)
    return path, count.to(torch.int32), token.to(torch.int32)


def _plain_accept(s, path, count):
    c, lens, page = s["case"], s["lens"].long(), s["case"]["page"]
    B, n = path.shape
    H = c["Hkv"]
    i = torch.arange(n, device=path.device)
    base = lens - n
    moves = (i < count[:, None]) & (path > i)
    b, i = torch.nonzero(moves, as_tuple=True)
    src, dst = base[b] + path[b, i], base[b] + i
    first = (base + (path == torch.arange(n, device=path.device)).sum(1))[b]  # the first slot that receives
    from_, to = s["table"][b, src // page].long(), s["table"][b, dst // page].long()
    for pool, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        kind, P = pool.dtype, pool.shape[0]
        rows = to[:, None].expand(-1, H)
        new = torch.zeros(P, H, device=path.device).scatter_reduce(0, rows, scale[from_], "amax")
        held = torch.zeros(P, dtype=torch.long, device=path.device).scatter_reduce(0, to, (first - dst // page * page).clamp(0, page), "amax")
        gets = torch.zeros(P, dtype=torch.bool, device=path.device).index_fill(0, to, True)
        new = torch.where((held > 0)[:, None], torch.maximum(new, scale), new)
        new = torch.where(gets[:, None], new, scale)
        x = _round8(pool[from_, :, src % page].float() * (scale[from_] / new[to])[..., None], kind)
        grown = torch.nonzero(gets[:, None] & (held > 0)[:, None] & (new > scale), as_tuple=True)
        blocks = pool[grown].float() * (scale[grown] / new[grown])[:, None, None]
        live = torch.arange(page, device=path.device) < held[grown[0]][:, None]
        _bytes(pool)[grown] = torch.where(live[..., None], _bytes(_round8(blocks, kind)), _bytes(pool)[grown])
        _bytes(pool)[to, :, dst % page] = _bytes(x)
        scale.copy_(new)
    if "weights" in s:
        w = s["weights"]
        w[b, :, dst] = w[b, :, src]
    return (base + count).to(torch.int32)


def run(state):
    s, c = state, state["case"]
    op, opt = c["op"], {k: c[k] for k in ("softcap", "window") if k in c}
    if own:
        import attention_forward_08_gb300 as fa
        if op == "step":
            fa.cache_append(s["cache"], s["new_k"], s["new_v"], s["table"], s["before"], weights=s.get("weights"))
        if op in ("attn", "step"):
            o, lse = fa.cache_attention(s["q"], s["cache"], s["table"], s["lens"], tree=s["tree"],
                                        weights=s.get("weights"), **opt)
        if op in ("verify", "step"):
            path, count, token = fa.verify_drafts(s["p"], s["tokens"], s["tree"], s["u"], s["u_next"],
                                                  p_draft=s.get("p_draft"))
        if op == "accept":
            path, count = s["path"], s["count"]
        if op in ("accept", "step"):
            lens = fa.cache_accept(s["cache"], s["table"], s["lens"], path, count, weights=s.get("weights"))
    else:
        if op == "step":
            _plain_append(s["k"], s["ks"], s["new_k"], s["table"], s["before"])
            _plain_append(s["v"], s["vs"], s["new_v"], s["table"], s["before"])
            if "weights" in s:  # new slots start without weight
                at = s["before"].long()[:, None] + torch.arange(c["n"], device=DEV)
                s["weights"].scatter_(2, at[:, None].expand(-1, c["Hkv"], -1), 0.0)
        if op in ("attn", "step"):
            o, lse = _plain_attention(s)
        if op in ("verify", "step"):
            path, count, token = _plain_verify(s)
        if op == "accept":
            path, count = s["path"], s["count"]
        if op in ("accept", "step"):
            lens = _plain_accept(s, path, count)
    out = {}
    if op in ("attn", "step"):
        out.update(o=o, lse=lse)
    if op in ("verify", "step"):
        out.update(path=path, count=count, token=token)
    if op in ("accept", "step"):
        out.update(k=s["k"], v=s["v"], k_scale=s["ks"], v_scale=s["vs"], lens=lens)
    if "weights" in s:
        out["weights"] = s["weights"]
    return out


# ---------------------------------------------------------------- the definition, in 64 bits


def _exact_attention(s):
    """Sequence by sequence and node by node over the slots that it sees."""
    c, q = s["case"], s["q"]
    B, Hq, n, D = q.shape
    H, page = c["Hkv"], c["page"]
    cap, window = c.get("softcap", 0.0), c.get("window", 0)
    o = torch.zeros(B, Hq, n, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Hq, n, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if "weights" in s else None
    trees = s["tree"].expand(B, n).tolist()
    for b, L in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-L // page)].long()
        take = lambda x, y: (x[pages].double() * y[pages].double()[:, :, None, None]).transpose(0, 1).reshape(H, -1, D)[:, :L]  # noqa: E731
        k, v = take(s["k"], s["ks"]), take(s["v"], s["vs"])
        hidden = torch.ones(n, L, dtype=torch.bool)
        for i in range(n):
            line, a = [], i  # the way up
            while a >= 0:
                line.append(a)
                a = trees[b][a]
            line = line[:window] if window else line
            lo = max(0, L - n + len(line) - window) if window and len(line) < window else 0
            if not window or len(line) < window:
                hidden[i, lo:L - n] = False
            hidden[i, [L - n + a for a in line]] = False
        hidden = hidden.to(DEV)
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


def _exact_verify(s):
    """Request by request, down the tree: at each node its children in turn."""
    B, n, V = s["p"].shape
    tokens, u, after = s["tokens"].tolist(), s["u"].tolist(), s["u_next"].tolist()
    path, count, token = torch.full((B, n), -1, dtype=torch.int32), [], []
    for b, tree in enumerate(s["tree"].expand(B, n).tolist()):
        line, more = [0], True
        while more:
            more, at = False, line[-1]
            have, rounds = s["p"][b, at].double(), 1.0
            less = s["p_draft"][b, at].double() if "p_draft" in s else None
            for i in range(at + 1, n):
                if tree[i] != at:
                    continue
                t = tokens[b][i]
                if u[b][i] * rounds * (1.0 if less is None else float(less[t])) < float(have[t]):
                    line.append(i)
                    more = True
                    break
                if less is None:
                    rounds -= float(have[t])
                    have = have.clone()
                    have[t] = 0.0
                else:
                    have = torch.relu(have - rounds * less)
                    rounds = float(have.sum())
        if not float(have.sum()) > 0.0:
            have = s["p"][b, line[-1]].double()
        upto = torch.cumsum(have, 0)
        token.append(int(torch.searchsorted(upto, after[b] * upto[-1:], right=True)))
        count.append(len(line))
        path[b, :len(line)] = torch.tensor(line, dtype=torch.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return path.to(DEV), i32(count), i32(token)


def _exact_round(x, kind):
    """To the nearest value of the type, ties to even, on its grid."""
    top = _top(kind)[2]
    x = x.clamp(-top, top)
    if kind == I8:
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_accept(s):
    """Request by request and block by block."""
    page, got = s["case"]["page"], {}
    counts = s["count"].tolist()
    n = s["path"].shape[1]
    for name in ("k", "v"):
        kind, pool, scale = s[name].dtype, s[name].double(), s[name + "s"].double()
        for b, L in enumerate(s["lens"].tolist()):
            blocks, line = s["table"][b].tolist(), s["path"][b].tolist()
            kept = [L - n + a for a in line[:counts[b]]]  # the slot whose token comes to base + i
            for m in range((L - n) // page, (L - n + counts[b] - 1) // page + 1):
                lo, hi = max(L - n, m * page), min(L - n + counts[b], (m + 1) * page)
                src = list(range(m * page, lo)) + kept[lo - (L - n):hi - (L - n)]
                if src == list(range(m * page, hi)):
                    continue
                at, rows = [blocks[j // page] for j in src], [j % page for j in src]
                top = scale[at].amax(0)
                x = _exact_round(pool[at, :, rows] * (scale[at] / top)[..., None], kind)
                pool[blocks[m], :, :hi - m * page] = x.transpose(0, 1)
                scale[blocks[m]] = top
        got[name], got[name + "_scale"] = pool if kind == E4M3 else None, scale
    return dict(got, lens=s["lens"] - n + s["count"])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "accept":
        return dict(_exact_accept(s), **({"weights": None} if "weights" in s else {}))
    if case["op"] == "verify":
        path, count, token = _exact_verify(s)
        return dict(path=path, count=count, token=token)
    out = {}
    if case["op"] == "step":  # whole pools of stored values: the attention reads what was written
        _plain_append(s["k"], s["ks"], s["new_k"], s["table"], s["before"])
        _plain_append(s["v"], s["vs"], s["new_v"], s["table"], s["before"])
        if "weights" in s:
            for b, L in enumerate(s["before"].tolist()):
                s["weights"][b, :, L:L + case["n"]] = 0.0
    o, lse, weights = _exact_attention(s)
    out.update(o=o, lse=lse)
    if case["op"] == "step":
        path, count, token = _exact_verify(s)
        out.update(path=path, count=count, token=token, k=None, v=None, k_scale=None, v_scale=None, lens=s["before"] + count)
        weights = None  # (they move along the path)
    if "weights" in s:
        out["weights"] = weights
    return out
