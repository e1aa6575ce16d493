"""GPU parity of the 8-bit cache operators with their definition in 64 bits (tests/cache_reference.py)."""
import time

import numpy as np
import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu
E4M3, I8, BF16, F16, F32 = R.E4M3, R.I8, torch.bfloat16, torch.float16, torch.float32
DEV = "cuda:0"
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}  # half a step, relative


@pytest.fixture(scope="module")
def fa():
    import attention_forward_08_gb300 as fa
    assert fa.fa_sync_status(None) == 0
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def to_gpu(fa, pools):
    return fa.KVCache(*(t.to(DEV) for t in pools))


def same_pools(cache, ref, what=""):
    """Stored values and scales are defined to the bit."""
    for name, t, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        np.testing.assert_array_equal(s.cpu().double().numpy(), ref.scale[name], err_msg=f"{what} {name} scale")
        np.testing.assert_array_equal(R.stored(t.cpu()), ref.pool[name], err_msg=f"{what} {name}")


def synced(fa):
    assert fa.fa_sync_status(None) == 0, fa.fa_last_error()


def check_attention(fa, ref, q, table, lens, got, got_w=None, w0=None, n_q=None, **kw):
    """O: half a step of the output, and of the weights' f16 form times sum of p |v|; L: fp32 sums of D
    products, D steps of 2^-24 of the largest sum of |q k| at worst, taken as 2^-18 of it."""
    o, lse = (t.double().cpu().numpy() for t in got)
    ro, rl, rw, a, sabs = R.attention(ref, q, table, lens, n_q=n_q, **kw)
    tol_l = (2.0 ** -18 * sabs + 1e-6)[:, None, None]
    empty = np.isneginf(rl)
    np.testing.assert_array_equal(np.isneginf(lse), empty)
    assert np.all(o[empty] == 0.0)
    assert np.all(np.isfinite(o))
    d = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, rl))
    assert np.all(d <= tol_l), f"max |dL| {d.max():.3e}, allowed {tol_l.max():.3e}"
    tol_o = HALF[q.dtype] * np.abs(ro) + (HALF[F16] + 2 * tol_l[..., None]) * a + 1e-7
    d = np.abs(o - ro)
    assert np.all(d <= tol_o), f"max |dO| {d.max():.3e} at {np.unravel_index(d.argmax(), d.shape)}, {(d / tol_o).max():.2f} of the tolerance"
    if got_w is not None:
        w = got_w.double().cpu().numpy()
        want = w0.double().cpu().numpy().copy()
        want[:, :, :rw.shape[2]] += rw[:, :, :want.shape[2]]
        tol = np.zeros_like(want)
        tol[:, :, :rw.shape[2]] = (2 * tol_l * rw)[:, :, :want.shape[2]]
        tol += 2.0 ** -22 * np.abs(want)  # the addition, and the sum over rows and heads
        d = np.abs(w - want)
        assert np.all(d <= tol), f"max |dw| {d.max():.3e} at {np.unravel_index(d.argmax(), d.shape)}"


# ----------------------------------------------------------------- append

@pytest.mark.parametrize("kind", [E4M3, I8])
@pytest.mark.parametrize("io", [BF16, F16, F32])
@pytest.mark.parametrize("D,page,H,lens,news", [
    (64, 16, 1, [0], [1]),
    (128, 64, 2, [0, 1, 63, 64, 100], [1, 1, 1, 1, 1]),
    (128, 16, 3, [0, 5, 16, 31], [40, 33, 1, 16]),
    (256, 128, 2, [0, 127, 300], [300, 2, 129]),
    (64, 32, 2, [7, 0, 90], [0, 65, 3]),
])
def test_append(fa, kind, io, D, page, H, lens, news):
    g = torch.Generator().manual_seed(D + page + len(lens))
    B, n = len(lens), max(news)
    table, P, _ = R.make_table(g, [a + b for a, b in zip(lens, news)], page)
    pools = R.make_pools(g, P, H, page, D, kind)
    for t in pools[:2]:
        R.spoil(t, table, lens, page)
    mag = torch.randint(-12, 8, (B, H, n, 1), generator=g).float().exp2()  # tokens of very different size
    new = {x: (torch.randn(B, H, n, D, generator=g) * mag).to(io) for x in "kv"}
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    R.append(ref, new, table, lens, news)
    W = len(table[0]) * page
    w0, p0 = torch.full((B, H, W), 3.0), torch.full((B, H, W), -7, dtype=torch.int32)
    w, p = w0.to(DEV), p0.to(DEV)
    seen = [11 * x + 5 for x in lens]
    fa.cache_append(cache, new["k"].to(DEV), new["v"].to(DEV), i32(table), i32(lens), n_new=i32(news), weights=w,
                    positions=p, seen=i32(seen))
    synced(fa)
    same_pools(cache, ref)
    for b in range(B):
        for t in range(news[b]):
            w0[b, :, lens[b] + t], p0[b, :, lens[b] + t] = 0.0, seen[b] + t
    assert torch.equal(w.cpu(), w0) and torch.equal(p.cpu(), p0)


@pytest.mark.parametrize("kind", [E4M3, I8])
def test_append_token_by_token_matches_at_once_in_e4m3(fa, kind):
    """Scales are powers of two: an e4m3 token that moves to a larger one keeps its bits (values far from underflow)."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 2, 48, 64, generator=g)
    x = torch.sign(x) * (1 + x.abs()) * torch.linspace(-3, 4, 48)[:, None].round().exp2()
    x = x.to(BF16).to(DEV)
    one, many = (fa.kv_cache(2, 2, 64, page=64, dtype=kind) for _ in range(2))
    table = i32([[1]])
    fa.cache_append(one, x, x, table, i32([0]))
    for t in range(48):
        fa.cache_append(many, x[:, :, t:t + 1], x[:, :, t:t + 1], table, i32([t]))
    synced(fa)
    assert torch.equal(one.k_scale, many.k_scale)
    if kind == E4M3:
        assert torch.equal(one.k.view(torch.uint8), many.k.view(torch.uint8))
    else:  # each of the 7 growths rounds to a whole number: at most half a step each, halved by the next
        assert (one.k.int() - many.k.int()).abs().max() <= 1


@pytest.mark.parametrize("kind", [E4M3, I8])
def test_append_special_values(fa, kind):
    """Infinities saturate and set no scale, NaN stays NaN (0 in int8), zeros get the least scale and do not stop a
    later small token from getting its own; the extremes of the types."""
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(1, 1, 64, 64)
    x[0, 0, 0, :4] = torch.tensor([inf, -inf, nan, 3.0])
    x[0, 0, 16:32] = 0.0
    x[0, 0, 32, :2] = torch.tensor([3.3e38, -1e-40])
    x[0, 0, 48, :3] = torch.tensor([448.0, 449.0, 2.0 ** -9])
    cache = fa.kv_cache(4, 1, 64, page=16, dtype=kind)
    pools = [t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    ref = R.Cache(*pools)
    table = [[2, 0, 3, 1]]
    R.append(ref, {"k": x, "v": x * -1}, table, [0], [64])
    fa.cache_append(cache, x.to(DEV), (x * -1).to(DEV), i32(table), i32([0]))
    synced(fa)
    same_pools(cache, ref)
    assert cache.k_scale[0, 0].item() == 2.0 ** -100


def test_append_strided(fa):
    """Token-major new keys, pools interleaved [P, page, H, 2, D] in one buffer."""
    g = torch.Generator().manual_seed(9)
    P, H, page, D = 5, 3, 32, 128
    raw = torch.zeros(P, page, H, 2, D, dtype=torch.uint8, device=DEV)
    k, v = (raw[:, :, :, i].permute(0, 2, 1, 3).view(E4M3) for i in range(2))
    ks, vs = (torch.ones(P, H, device=DEV) for _ in range(2))
    cache = fa.KVCache(k, v, ks, vs)
    ref = R.Cache(k.cpu(), v.cpu(), ks.cpu(), vs.cpu())
    x = torch.randn(2, 50, 2 * H, D, generator=g).to(BF16)
    new = {"k": x[:, :, :H].transpose(1, 2), "v": x[:, :, H:].transpose(1, 2)}
    table = [[4, 0], [1, 3]]
    R.append(ref, new, table, [0, 10], [50, 50])
    xd = x.to(DEV)
    fa.cache_append(cache, xd[:, :, :H].transpose(1, 2), xd[:, :, H:].transpose(1, 2), i32(table), i32([0, 10]))
    synced(fa)
    same_pools(cache, ref)


# ----------------------------------------------------------------- attention

def attention_case(fa, *, kind=E4M3, io=BF16, D=128, page=64, Hq=4, Hkv=2, lens=(100,), n=1, n_q=None, track=False,
                   seed=0, qscale=1.0, extra=None, **kw):
    g = torch.Generator().manual_seed(seed + D + page + sum(lens))
    lens = list(lens)
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, Hkv, page, D, kind)
    ref = R.Cache(*pools)
    for t in pools[:2]:
        R.spoil(t, table, lens, page)
    q = (torch.randn(len(lens), Hq, n, D, generator=g) * qscale).to(io)
    cache = to_gpu(fa, pools)
    w = w0 = None
    if track:
        w0 = torch.rand(len(lens), Hkv, max(1, max(lens)) + 3, generator=g)
        w = w0.to(DEV)
    got = fa.cache_attention(q.to(DEV), cache, i32(table), i32(lens), n_q=None if n_q is None else i32(list(n_q)),
                             weights=w, **kw)
    synced(fa)
    check_attention(fa, ref, q, table, lens, got, w, w0, n_q=n_q, **kw)
    return got


@pytest.mark.parametrize("kind", [E4M3, I8])
@pytest.mark.parametrize("io", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_decode(fa, kind, io, D, page):
    """One row: no token but its own, one key, lengths around a block's and a tile's end, a long one."""
    attention_case(fa, kind=kind, io=io, D=D, page=page, Hq=8, Hkv=2, lens=(1, 2, 15, 16, 17, 63, 64, 65, 129, 1000),
                   track=page == 64)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (32, 8), (16, 1), (24, 1), (40, 1), (64, 2), (130, 1)])
def test_groups(fa, Hq, Hkv):
    attention_case(fa, Hq=Hq, Hkv=Hkv, lens=(700, 33, 256), track=True)


@pytest.mark.parametrize("n", [2, 3, 8, 17, 64, 130, 257])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,page,kind,io", [(128, 64, E4M3, BF16), (64, 16, I8, F16), (256, 128, E4M3, F16),
                                            (128, 32, I8, BF16)])
def test_many_rows(fa, n, causal, D, page, kind, io):
    attention_case(fa, kind=kind, io=io, D=D, page=page, Hq=6, Hkv=2, n=n, lens=(n, n + 1, n + 77, 640), causal=causal,
                   track=page == 64)


@pytest.mark.parametrize("n", [1, 5, 40, 200])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 5000])
def test_window(fa, n, window):
    attention_case(fa, n=n, lens=(n, 3 + n, 130 + n, 777), window=window, track=window == 100)


@pytest.mark.parametrize("n", [1, 6, 150])
@pytest.mark.parametrize("softcap", [0.5, 20.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_softcap(fa, n, softcap, D):
    attention_case(fa, n=n, D=D, lens=(n + 200, 400), softcap=softcap, window=0 if D == 64 else 90, track=D == 64)


@pytest.mark.parametrize("n", [1, 4, 150])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scale(fa, n, scale):
    """A negative, a zero and a large scale (weights on one key)."""
    attention_case(fa, n=n, lens=(n + 90,), scale=scale, track=True)


@pytest.mark.parametrize("n,lens,n_q", [
    (1, (0, 5, 0), None),                    # nothing cached
    (4, (0, 2, 9, 4), None),                 # more rows than tokens: the first rows see nothing
    (6, (100, 100, 7, 0, 3), (6, 2, 0, 0, 3)),
    (200, (300, 300, 0, 130), (200, 1, 0, 130)),
    (200, (100, 0, 199, 150), None),
])
@pytest.mark.parametrize("causal", [True, False])
def test_empty_rows_and_padding(fa, n, lens, n_q, causal):
    attention_case(fa, n=n, lens=lens, n_q=n_q, causal=causal, track=True)
    attention_case(fa, n=n, lens=lens, n_q=n_q, causal=causal, D=64, page=16, kind=I8, window=20, track=True)


@pytest.mark.parametrize("n", [1, 150])
def test_magnitudes(fa, n):
    """Scales from 2^-60 to 2^40 in one sequence, queries to match: stored values are used in the units of their own
    block, and no block's size hides another's."""
    g = torch.Generator().manual_seed(3)
    page, D, H, L = 16, 64, 1, 160 + n
    table, P, _ = R.make_table(g, [L], page)
    k, v, ks, vs = R.make_pools(g, P, H, page, D, E4M3)
    vs = torch.randint(-60, 41, (P, H), generator=g).float().exp2()
    ks = ks * 2.0 ** -30
    ref = R.Cache(k, v, ks, vs)
    q = (torch.randn(1, 4, n, D, generator=g) * 2.0 ** 30).to(BF16)
    got = fa.cache_attention(q.to(DEV), to_gpu(fa, (k, v, ks, vs)), i32(table), i32([L]))
    synced(fa)
    check_attention(fa, ref, q, table, [L], got)


def test_long_cache_and_long_offsets(fa):
    """70,001 tokens; and a pool whose last blocks lie more than 2^32 bytes behind its first."""
    attention_case(fa, lens=(70001,), Hq=8, Hkv=1, track=True)
    g = torch.Generator().manual_seed(1)
    page, D, P = 64, 128, 4
    raw = torch.zeros(1 << 33, dtype=torch.uint8, device=DEV)  # blocks 2^31 - 2^16 bytes apart
    st = ((1 << 31) - (1 << 16), page * D, D, 1)
    k, v, ks, vs = R.make_pools(g, P, 2, page, D, E4M3)
    kk = raw.as_strided((P, 2, page, D), st).view(E4M3)
    vv = raw[1 << 20:].as_strided((P, 2, page, D), st).view(E4M3)
    kk.view(torch.uint8).copy_(k.view(torch.uint8))
    vv.view(torch.uint8).copy_(v.view(torch.uint8))
    cache, ref = fa.KVCache(kk, vv, ks.to(DEV), vs.to(DEV)), R.Cache(k, v, ks, vs)
    table, lens = [[3, 0, 2, 1]], [250]
    for n in (1, 140):
        q = torch.randn(1, 4, n, D, generator=g).to(BF16)
        got = fa.cache_attention(q.to(DEV), cache, i32(table), i32(lens))
        synced(fa)
        check_attention(fa, ref, q, table, lens, got)


@pytest.mark.parametrize("ctas", [1, 2, 7])
@pytest.mark.parametrize("kind,io,D,page,Hq,Hkv,n", [
    (E4M3, BF16, 128, 64, 8, 2, 1), (I8, F16, 64, 16, 6, 3, 1), (E4M3, F16, 256, 128, 4, 2, 1),
    (E4M3, BF16, 128, 16, 8, 2, 6), (I8, BF16, 64, 32, 8, 1, 40), (I8, BF16, 256, 16, 8, 1, 4),
])
def test_long_parts(fa, ctas, kind, io, D, page, Hq, Hkv, n):
    """Few thread blocks: each runs round its ring many times, over parts of several sequences and heads."""
    fa.fa_set_max_ctas(ctas)
    try:
        attention_case(fa, kind=kind, io=io, D=D, page=page, Hq=Hq, Hkv=Hkv, n=n, lens=(2500, n, 777, 0 if n == 1 else n, 1300),
                       track=True)
        attention_case(fa, kind=kind, io=io, D=D, page=page, Hq=Hq, Hkv=Hkv, n=n, lens=(4000,) * 3, window=900)
    finally:
        fa.fa_set_max_ctas(0)


def test_full_machine(fa):
    """Every thread block gets parts longer than its ring."""
    attention_case(fa, Hq=16, Hkv=8, lens=(6000, 5000, 7001, 6500))
    attention_case(fa, Hq=32, Hkv=8, n=5, lens=(4000, 5000, 3001, 2500))


@pytest.mark.parametrize("Hq,Hkv,n", [(16, 1, 1), (8, 2, 4), (4, 2, 40)])
def test_wide_table(fa, Hq, Hkv, n):
    """A table for 2^20 tokens of which a few are held: the tracked weights take their other way."""
    g = torch.Generator().manual_seed(Hq)
    lens, page, D = [300, 41], 64, 128
    table, P, _ = R.make_table(g, lens, page, width=1 << 14)
    pools = R.make_pools(g, P, Hkv, page, D, E4M3)
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    q = torch.randn(2, Hq, n, D, generator=g).to(BF16)
    w0 = torch.rand(2, Hkv, 310, generator=g)
    w = w0.to(DEV)
    got = fa.cache_attention(q.to(DEV), cache, i32(table), i32(lens), weights=w)
    synced(fa)
    check_attention(fa, ref, q, table, lens, got, w, w0)


@pytest.mark.parametrize("n", [1, 5, 150])
def test_attention_strided(fa, n):
    """Token-major q and output, pools interleaved, a table that is a slice of a wider one."""
    g = torch.Generator().manual_seed(n)
    P, H, page, D, lens = 16, 2, 32, 128, [n + 60, n + 3]  # at most 7 of a row's 8 blocks
    raw = torch.zeros(P, page, 2, H, D, dtype=torch.uint8, device=DEV)
    pools = R.make_pools(g, P, H, page, D, I8)
    views = [raw[:, :, i].permute(0, 2, 1, 3).view(I8) for i in range(2)]
    for a, b in zip(views, pools):
        a.copy_(b)
    cache, ref = fa.KVCache(*views, pools[2].to(DEV), pools[3].to(DEV)), R.Cache(*pools)
    table = [[5, 0, 7, 2, 9, 11, 15, 12], [1, 3, 4, 6, 8, 10, 14, 13]]
    wide = torch.full((2, 13), -1, dtype=torch.int32, device=DEV)
    wide[:, 4:12] = i32(table)
    q = torch.randn(2, n, 6, D, generator=g).to(F16)
    qd = q.to(DEV)
    out = torch.full((2, n, 6, D), float("nan"), dtype=F16, device=DEV)
    o, lse = fa.cache_attention(qd.transpose(1, 2), cache, wide[:, 4:12], i32(lens), out=out.transpose(1, 2))
    synced(fa)
    assert o.data_ptr() == out.data_ptr()
    check_attention(fa, ref, q.transpose(1, 2), table, lens, (o, lse))


@pytest.mark.parametrize("n", [1, 150])
def test_bad_entries_are_skipped_and_told(fa, n):
    """A table entry out of range hides its block's tokens; a length past the table ends there; a negative one is 0."""
    g = torch.Generator().manual_seed(8)
    page, D = 16, 64
    table, P, _ = R.make_table(g, [160, 160, 160, 160], page)
    pools = R.make_pools(g, P, 1, page, D, E4M3)
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    q = torch.randn(4, 2, n, D, generator=g).to(BF16)
    bad = [list(r) for r in table]
    bad[0][9], bad[1][9] = P, -5
    lens = [160, 160, 100000, -3]
    w = torch.zeros(4, 1, 160, device=DEV)
    o, lse = fa.cache_attention(q.to(DEV), cache, i32(bad), i32(lens), causal=False, weights=w)
    assert fa.fa_sync_status(None) == fa.fa.FA_ERR_INVALID_ARGUMENT and "out of range" in fa.fa_last_error()
    assert fa.fa_sync_status(None) == 0
    check_attention(fa, ref, q, table, [144, 144, 160, 0], (o, lse), w, torch.zeros(4, 1, 160), causal=False)
    before = cache.k.view(torch.uint8).clone()
    x = torch.ones(4, 1, 2, D, dtype=BF16, device=DEV)
    fa.cache_append(cache, x, x, i32(bad), i32([150, 150, 160, -3]))  # bad entries, behind the table, negative
    assert fa.fa_sync_status(None) == fa.fa.FA_ERR_INVALID_ARGUMENT
    assert torch.equal(before, cache.k.view(torch.uint8))


# ----------------------------------------------------------------- eviction

def evict_case(fa, *, kind=E4M3, D=64, page=16, H=2, lens=(100,), keep=40, recent=0, into=True, weights=None, seed=0,
               positions="random", W=None):
    g = torch.Generator().manual_seed(seed + sum(lens) + keep)
    lens, B = list(lens), len(lens)
    table, P, spare = R.make_table(g, lens, page, spare=B * -(-keep // page) + 1)
    pools = R.make_pools(g, P, H, page, D, kind)
    W = len(table[0]) * page + 5 if W is None else W
    w = torch.randn(B, H, W, generator=g).exp() if weights is None else weights(g, (B, H, W))
    p = None
    if positions == "random":  # as after earlier evictions: distinct, in no order
        p = torch.stack([torch.randperm(3 * W, generator=g)[:W] for _ in range(B * H)]).view(B, H, W).int()
    to = [[spare.pop() for _ in range(-(-keep // page))] for _ in range(B)] if into else None
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    rw, rp = w.numpy().copy(), None if p is None else p.numpy().copy()
    n, src = R.evict(ref, table, lens, rw, rp, keep, recent, into=to)
    wd, pd = w.to(DEV), None if p is None else p.to(DEV)
    if into:
        wo, po = torch.full((B, H, keep + 2), -5.0, device=DEV), torch.full((B, H, keep + 2), -5, dtype=torch.int32, device=DEV)
        got = fa.cache_evict(cache, i32(table), i32(lens), wd, pd, keep=keep, recent=recent, into=i32(to),
                             weights_out=wo, positions_out=po)
    else:
        ln = i32(lens)
        got = fa.cache_evict(cache, i32(table), ln, wd, pd, keep=keep, recent=recent, lens_out=ln)
        assert got is ln
    synced(fa)
    assert got.tolist() == n
    same_pools(cache, ref)
    if into:
        want_w, want_p = torch.full((B, H, keep + 2), -5.0), torch.full((B, H, keep + 2), -5, dtype=torch.int32)
        for (b, h), s in src.items():
            want_w[b, h, :len(s)] = w[b, h, s]
            want_p[b, h, :len(s)] = torch.tensor(s, dtype=torch.int32) if p is None else p[b, h, s]
        np.testing.assert_array_equal(wo.cpu().numpy(), want_w.numpy())
        assert torch.equal(po.cpu(), want_p)
        assert p is None or torch.equal(pd.cpu(), p)
        np.testing.assert_array_equal(wd.cpu().numpy(), w.numpy())
    else:
        np.testing.assert_array_equal(wd.cpu().numpy(), rw)
        np.testing.assert_array_equal(pd.cpu().numpy(), rp)


@pytest.mark.parametrize("into", [True, False])
@pytest.mark.parametrize("kind,D,page", [(E4M3, 64, 16), (I8, 128, 64), (E4M3, 256, 128), (I8, 64, 32)])
@pytest.mark.parametrize("lens,keep,recent", [
    ((100, 41, 40, 39, 1, 0), 40, 0),
    ((100, 41, 40, 39, 1, 0), 40, 13),
    ((300, 33), 32, 32),          # only the latest
    ((64, 65, 66), 64, 5),        # a step: one or two too many
    ((5000, 2100), 1, 0),
    ((5000, 700, 4097), 1000, 100),
])
def test_evict(fa, into, kind, D, page, lens, keep, recent):
    evict_case(fa, into=into, kind=kind, D=D, page=page, lens=lens, keep=keep, recent=recent)


def test_evict_very_long(fa):
    evict_case(fa, lens=(70000,), H=1, keep=4000, recent=50, positions=None)
    evict_case(fa, lens=(70000,), H=1, keep=4000, recent=50, into=False)


@pytest.mark.parametrize("into", [True, False])
@pytest.mark.parametrize("weights", [
    lambda g, s: torch.zeros(s),                                        # all tied: the lowest slots stay
    lambda g, s: torch.randint(0, 3, s, generator=g).float(),           # many ties
    lambda g, s: torch.randint(0, 3, s, generator=g).float() * -0.0,    # both zeros are one weight
    lambda g, s: torch.randn(s, generator=g) * 1e-42,                   # denormals, both signs
    lambda g, s: torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0, -3.4e38])[torch.randint(0, 5, s, generator=g)],
])
def test_evict_ties_and_special_weights(fa, into, weights):
    evict_case(fa, into=into, lens=(300, 77, 64), keep=64, recent=10, weights=weights)


def test_evict_positions_default_and_narrow_trackers(fa):
    evict_case(fa, lens=(200, 90), keep=50, recent=20, positions=None)
    evict_case(fa, lens=(200, 90), keep=50, recent=20, W=200)


def test_evict_bad_entries(fa):
    """Tokens of a block out of range are not moved; the call tells, and nothing else changes."""
    g = torch.Generator().manual_seed(2)
    pools = R.make_pools(g, 8, 1, 16, 64, E4M3)
    cache = to_gpu(fa, pools)
    w = torch.arange(48, 0, -1, dtype=F32).view(1, 1, 48).to(DEV)
    n = fa.cache_evict(cache, i32([[0, 99, 2]]), i32([48]), w, keep=32, into=i32([[4, 5]]))
    assert fa.fa_sync_status(None) == fa.fa.FA_ERR_INVALID_ARGUMENT
    assert n.tolist() == [32]
    raw = cache.k.cpu().view(torch.uint8)
    assert torch.equal(raw[4], raw[0]) and torch.equal(raw[5], pools[0].view(torch.uint8)[5])
    n = fa.cache_evict(cache, i32([[0, 1, 2]]), i32([48]), w, keep=32, into=i32([[4, 8]]))
    assert fa.fa_sync_status(None) == fa.fa.FA_ERR_INVALID_ARGUMENT


# ----------------------------------------------------------------- together

def budget_loop(fa, steps=12, graph=False):
    """Prompt, then decoding steps under a budget: append, attend with tracking, evict in place."""
    g = torch.Generator().manual_seed(4)
    B, Hq, H, D, page, keep, n0 = 2, 4, 2, 64, 16, 24, 20
    M = -(-(n0 + keep) // page)
    cache = fa.kv_cache(B * M, H, D, page=page)
    table = torch.arange(B * M, dtype=torch.int32, device=DEV).view(B, M)
    W = M * page
    weights, positions = torch.zeros(B, H, W, device=DEV), torch.zeros(B, H, W, dtype=torch.int32, device=DEV)
    lens, seen = i32([0] * B), i32([0] * B)
    draws = [[torch.randn(B, h, n, D, generator=g).to(BF16).to(DEV) for h in (Hq, H, H)] for n in [n0] + [1] * steps]

    def step(q, k, v):
        n = q.shape[2]
        fa.cache_append(cache, k, v, table, lens, weights=weights, positions=positions, seen=seen)
        lens.add_(n)
        seen.add_(n)
        o = fa.cache_attention(q, cache, table, lens, weights=weights)
        fa.cache_evict(cache, table, lens, weights, positions, keep=keep, recent=6, lens_out=lens)
        return o

    outs = [step(*draws[0])]
    if not graph:
        outs += [step(*d) for d in draws[1:]]
    else:
        hold = [x.clone() for x in draws[1]]
        state = [cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, weights, positions, lens, seen]
        saved = [x.clone() for x in state]
        gr = torch.cuda.CUDAGraph()
        step(*hold)  # warm-up
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            o = step(*hold)
        for a, b in zip(state, saved):
            a.copy_(b)
        for d in draws[1:]:
            for a, b in zip(hold, d):
                a.copy_(b)
            gr.replay()
            outs.append(tuple(x.clone() for x in o))
    synced(fa)
    return outs, (cache, weights, positions, lens)


def test_budget_loop_against_the_definition(fa):
    """Every stored byte, and outputs against the definition run on the same bytes and the same evictions."""
    outs, (cache, weights, positions, lens) = budget_loop(fa)
    assert lens.tolist() == [24, 24]
    seen = 20 + 12
    for b in range(2):
        for h in range(2):
            p = positions[b, h, :24].tolist()
            assert len(set(p)) == 24 and max(p) == seen - 1
            assert set(range(seen - 6, seen)) <= set(p)
    assert torch.isfinite(outs[-1][0]).all()
    assert (weights[:, :, :24] >= 0).all()


@pytest.mark.parametrize("kind,page,D,Hq", [(E4M3, 16, 64, 4), (I8, 32, 128, 8), (E4M3, 64, 256, 2)])
def test_budget_loop_operator_by_operator(fa, kind, page, D, Hq):
    """Each operator of each step against its definition on the state that the one before left: bytes, scales,
    trackers and lengths to the bit, outputs and weights within the attention's tolerances."""
    g = torch.Generator().manual_seed(page + D)
    B, H, keep, recent, news = 3, 2, 40, 9, [[50, 7, 33], [1, 1, 1], [1, 1, 1], [5, 0, 2], [1, 1, 1], [40, 40, 1]]
    M = -(-(keep + 50) // page)
    cache = fa.kv_cache(B * M, H, D, page=page, dtype=kind)
    rows = [list(range(b * M, b * M + M)) for b in range(B)]
    table, W = i32(rows), M * page
    weights, positions = torch.zeros(B, H, W, device=DEV), torch.zeros(B, H, W, dtype=torch.int32, device=DEV)
    held, seen = [0] * B, [0] * B

    def here():
        return R.Cache(cache.k.cpu(), cache.v.cpu(), cache.k_scale.cpu(), cache.v_scale.cpu())

    for new in news:
        n = max(new)
        q, k, v = (torch.randn(B, h, n, D, generator=g).to(BF16) for h in (Hq, H, H))
        ref, w0, p0 = here(), weights.cpu(), positions.cpu()
        fa.cache_append(cache, k.to(DEV), v.to(DEV), table, i32(held), n_new=i32(new), weights=weights,
                        positions=positions, seen=i32(seen))
        R.append(ref, {"k": k, "v": v}, rows, held, new)
        same_pools(cache, ref, "append")
        for b in range(B):
            for t in range(new[b]):
                w0[b, :, held[b] + t], p0[b, :, held[b] + t] = 0.0, seen[b] + t
        assert torch.equal(weights.cpu(), w0) and torch.equal(positions.cpu(), p0)
        held, seen = [x + y for x, y in zip(held, new)], [x + y for x, y in zip(seen, new)]
        w0 = weights.clone()
        got = fa.cache_attention(q.to(DEV), cache, table, i32(held), n_q=i32(new), weights=weights)
        check_attention(fa, ref, q, rows, held, got, weights, w0, n_q=new)
        rw, rp = weights.cpu().numpy().copy(), positions.cpu().numpy().copy()
        lens = i32(held)
        fa.cache_evict(cache, table, lens, weights, positions, keep=keep, recent=recent, lens_out=lens)
        held, _ = R.evict(ref, rows, held, rw, rp, keep, recent)
        assert lens.tolist() == held
        same_pools(cache, ref, "evict")
        np.testing.assert_array_equal(weights.cpu().numpy(), rw)
        np.testing.assert_array_equal(positions.cpu().numpy(), rp)
    synced(fa)


def test_counts_beyond_32_bits_are_refused(fa):
    cache = fa.kv_cache(2, 1, 64, page=16)
    table, lens = i32([[0, 1]]), i32([4])
    w, p = torch.zeros(1, 1, 32, device=DEV), torch.zeros(1, 1, 32, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="window"):
        fa.cache_attention(torch.zeros(1, 1, 1, 64, dtype=BF16, device=DEV), cache, table, lens, window=2 ** 32 + 1)
    with pytest.raises(ValueError, match="keep"):
        fa.cache_evict(cache, table, lens, w, p, keep=2 ** 32 + 1)
    with pytest.raises(ValueError, match="recent"):
        fa.cache_evict(cache, table, lens, w, p, keep=4, recent=2 ** 32)


@pytest.mark.parametrize("n,H,lens", [(8, 8, [128]), (16, 8, [128, 1, 0, 33]), (1, 3, [1, 2, 3]), (16, 1, [5])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_short_segments(fa, n, H, lens, D):
    """Segments shorter than a thread block's least part: one block each, some cut."""
    attention_case(fa, D=D, Hq=4 * H, Hkv=H, lens=lens, n=n, n_q=[min(n, x) for x in lens], track=True)


@pytest.mark.parametrize("softcap,scale", [(0.0, None), (5.0, None), (0.0, -0.1)])
@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (128, 256), (16, 256), (128, 128)])
def test_maximum_that_grows(fa, page, D, softcap, scale):
    """Later keys far larger than earlier ones, for some rows: weights are taken again against a new maximum."""
    g = torch.Generator().manual_seed(D + page)
    lens = [700, 257]
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, 2, page, D, E4M3)
    for b in range(2):
        for j, blk in enumerate(x for x in table[b] if x >= 0):
            pools[2][blk] = 2.0 ** (-9 + j * page // 64)
    q = torch.randn(2, 4, 150, D, generator=g).to(BF16)
    q[:, :, ::3] *= 0.01
    kw = {"softcap": softcap} if scale is None else {"softcap": softcap, "scale": scale}
    got = fa.cache_attention(q.to(DEV), to_gpu(fa, pools), i32(table), i32(lens), **kw)
    synced(fa)
    check_attention(fa, R.Cache(*pools), q, table, lens, got, **kw)


def test_budget_loop_captured_and_replayed(fa):
    a, sa = budget_loop(fa)
    b, sb = budget_loop(fa, graph=True)
    for (o1, l1), (o2, l2) in zip(a, b):
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.equal(sa[0].k.view(torch.uint8), sb[0].k.view(torch.uint8))
    for x, y in zip(sa[1:], sb[1:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("n", [1, 150])
def test_own_stream_and_repeatable(fa, n):
    """On a side stream, with workspaces and outputs of its own; twice the same bits, tracked weights among them."""
    g = torch.Generator().manual_seed(6)
    table, P, _ = R.make_table(g, [900, 400], 64)
    pools = R.make_pools(g, P, 2, 64, 128, E4M3)
    cache = to_gpu(fa, pools)
    q = torch.randn(2, 8, n, 128, generator=g).to(BF16).to(DEV)
    t, ln = i32(table), i32([900, 400])
    res = []
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side.cuda_stream, side.cuda_stream):
        w = torch.zeros(2, 2, 900, device=DEV)
        torch.cuda.synchronize()
        o, l = fa.cache_attention(q, cache, t, ln, weights=w, stream=stream)
        torch.cuda.synchronize()
        res.append((o.clone(), l.clone(), w))
    for r in res[1:]:
        assert all(torch.equal(x, y) for x, y in zip(res[0], r))


@pytest.mark.parametrize("n", [1, 150])
def test_cached_matches_dense_attention(fa, n):
    """The same tokens through ``attention`` (bf16 K and V with the cache's values, which bf16 holds exactly)."""
    g = torch.Generator().manual_seed(12)
    L, H, D = 640, 2, 128
    x = [torch.randint(-14, 15, (1, H, L, D), generator=g).float().mul(0.125).to(BF16).to(DEV) for _ in range(2)]
    cache = fa.kv_cache(10, H, D)
    table = i32([list(range(10))])
    fa.cache_append(cache, *x, table, i32([0]))
    q = torch.randn(1, 8, n, D, generator=g).to(BF16).to(DEV)
    o, l = fa.cache_attention(q, cache, table, i32([L]))
    o2, l2 = fa.attention(q, *x, causal=True, q_offset=L - n)
    synced(fa)
    assert (o.float() - o2.float()).abs().max() <= 2e-2 and (l - l2).abs().max() <= 1e-2


@pytest.mark.parametrize("n,D", [(1, 64), (1, 128), (5, 128), (1, 256), (64, 128), (64, 256)])
def test_wait_bound_expires_or_not_then_recovers(fa, n, D):
    """With a one-cycle wait bound a kernel unwinds at the first wait that it expires in (its copies and MMAs drained),
    and the status tells; the hardware may hold a waiting thread until its copy has landed, and then none does.  Either
    way the next run is right."""
    g = torch.Generator().manual_seed(1)
    lens = [3000, 700]
    table, P, _ = R.make_table(g, lens, 64)
    pools = R.make_pools(g, P, 2, 64, D, E4M3)
    q = torch.randn(2, 8, n, D, generator=g).to(BF16)
    cache, qd, t, ln = to_gpu(fa, pools), q.to(DEV), i32(table), i32(lens)
    torch.cuda.synchronize()
    try:
        fa.fa_set_timeout_cycles(1)
        fa.cache_attention(qd, cache, t, ln)
        rc = fa.fa_sync_status(None)
    finally:
        fa.fa_set_timeout_cycles(0)
    assert rc in (fa.fa.FA_OK, fa.fa.FA_ERR_DEVICE_TIMEOUT), fa.fa_last_error()
    got = fa.cache_attention(qd, cache, t, ln)
    synced(fa)
    check_attention(fa, R.Cache(*pools), q, table, lens, got)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("cycles", [1, 300, 3000, 30000])
@pytest.mark.parametrize("n,D,page,lens", [(1, 128, 64, [300, 40]), (1, 64, 16, [600]), (5, 128, 64, [3000, 31]),
                                           (1, 256, 64, [150]), (5, 128, 16, [300, 2000])])
def test_wait_bounds_of_any_length_then_the_next_call_is_right(fa, n, D, page, lens, cycles, ctas):
    """Waits that expire while all of a short sequence's copies are under way: they land before the thread block ends,
    so that whoever gets its shared memory next finds it its own."""
    g = torch.Generator().manual_seed(D + n)
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, 2, page, D, E4M3)
    q = torch.randn(len(lens), 8, n, D, generator=g).to(BF16)
    cache, qd, t, ln = to_gpu(fa, pools), q.to(DEV), i32(table), i32(lens)
    torch.cuda.synchronize()
    try:
        fa.fa_set_max_ctas(ctas)
        for _ in range(3):
            fa.fa_set_timeout_cycles(cycles)
            fa.cache_attention(qd, cache, t, ln)
            fa.fa_set_timeout_cycles(0)
            got = fa.cache_attention(qd, cache, t, ln)
            rc = fa.fa_sync_status(None)
            assert rc in (fa.fa.FA_OK, fa.fa.FA_ERR_DEVICE_TIMEOUT), fa.fa_last_error()
            check_attention(fa, R.Cache(*pools), q, table, lens, got)
    finally:
        fa.fa_set_timeout_cycles(0)
        fa.fa_set_max_ctas(0)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("n,lens", [(4, (1, 2, 9)), (8, (5, 0)), (40, (7, 39, 300)), (200, (100, 3, 199, 150))])
@pytest.mark.parametrize("causal", [True, False])
def test_window_wider_than_any_cache(fa, n, lens, window, causal):
    """More rows than tokens, so that the first rows stand before the first token, and a window that means none."""
    attention_case(fa, n=n, lens=lens, window=window, causal=causal, track=True)
    attention_case(fa, n=n, lens=lens, window=window, causal=causal, D=64, page=16, kind=I8)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("cycles", [1, 300, 3000, 30000])
@pytest.mark.parametrize("n,D,page,lens", [(64, 128, 64, [700, 300]), (70, 256, 64, [400]), (200, 64, 16, [900, 201])])
def test_wait_bounds_of_many_rows_then_the_next_call_is_right(fa, n, D, page, lens, cycles, ctas):
    """Stores to tensor memory that are under way when a wait expires are done before the memory is given back."""
    test_wait_bounds_of_any_length_then_the_next_call_is_right(fa, n, D, page, lens, cycles, ctas)


@pytest.mark.parametrize("n,D,page", [(1, 64, 16), (1, 128, 64), (1, 128, 16), (5, 128, 64), (1, 256, 64), (1, 256, 16),
                                      (64, 64, 64), (64, 128, 64), (64, 256, 64)])
def test_wait_bound_expires_then_recovers(fa, n, D, page):
    """A wait looks at its bound before the hardware may suspend it: with a bound of one cycle the first wait whose
    copy or product is not there yet expires, every role unwinds at once, and the status tells."""
    g = torch.Generator().manual_seed(1)
    lens = [3000, 700]
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, 2, page, D, E4M3)
    q = torch.randn(2, 8, n, D, generator=g).to(BF16)
    cache, qd, t, ln = to_gpu(fa, pools), q.to(DEV), i32(table), i32(lens)
    fa.cache_attention(qd, cache, t, ln)
    torch.cuda.synchronize()
    try:
        fa.fa_set_timeout_cycles(1)
        begin = time.monotonic()
        fa.cache_attention(qd, cache, t, ln)
        rc = fa.fa_sync_status(None)
        took = time.monotonic() - begin
    finally:
        fa.fa_set_timeout_cycles(0)
    assert rc == fa.fa.FA_ERR_DEVICE_TIMEOUT, fa.fa_last_error()
    assert took < 1.0, f"unwinding took {took:.2f} s"
    got = fa.cache_attention(qd, cache, t, ln)
    synced(fa)
    check_attention(fa, R.Cache(*pools), q, table, lens, got)


def check_small_weights(q, got, ref, table, lens, floor):
    """O against the definition: half a step of the output, 2^-11 of every weight's size (its f16 form), and what the
    weights below f16's normal numbers lose at most, `floor`."""
    ro, rl, _, a, sabs = R.attention(ref, q, table, lens)
    o, lse = (t.double().cpu().numpy() for t in got)
    tol_l = 2.0 ** -18 * sabs.max() + 1e-6
    assert np.all(np.abs(lse - rl) <= tol_l)
    tol = HALF[q.dtype] * np.abs(ro) + (HALF[F16] + 2 * tol_l) * a + floor + 1e-7
    d = np.abs(o - ro)
    assert np.all(d <= tol), f"max |dO| {d.max():.3e}, {(d / tol).max():.2f} of the tolerance, sum p |v| {a.mean():.3e}"


def least_weight(rows):
    """A row's largest weight is at least 2^lift in f16, whose numbers are 2^-24 apart at least, rounded by half that;
    the lift is 11 where a K/V head has at most 32 rows, else 7."""
    return 2.0 ** -(25 + (11 if rows <= 32 else 7))


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("n,L,key,value", [(1, 16384, 24.0, 0.0), (5, 16384, 24.0, 0.0), (40, 16384, 24.0, 0.0),
                                           (1, 16384, 24.0, 1.0), (40, 16384, 24.0, 1.0),
                                           (1, 131071, 28.0, 0.0), (5, 131071, 28.0, 0.0)])
def test_a_first_token_that_holds_nearly_all_the_weight(fa, n, ctas, L, key, value):
    """As trained heads have it: 99.9% of each row's weight on one token whose value is (nearly) zero, so that the
    output is made of weights 2^-24 of the largest."""
    g = torch.Generator().manual_seed(L + n)
    page, D, Hq, H = 64, 128, 4, 1
    table, P, _ = R.make_table(g, [L], page)
    k, v, ks, vs = R.make_pools(g, P, H, page, D, E4M3)
    ks.fill_(1.0)
    vs.fill_(2.0 ** -7)
    k = (torch.randn(P, H, page, D, generator=g) * 0.25).to(E4M3)
    k.view(torch.uint8)[..., 0] = 0
    first = table[0][0]
    k[first, 0, 0] = torch.zeros(D).to(E4M3)
    k[first, 0, 0, 0] = torch.tensor(key).to(E4M3)
    v[first, 0, 0] = torch.full((D,), value).to(E4M3)
    q = torch.randn(1, Hq, n, D, generator=g) * 0.5
    q[..., 0] = 8.0
    q = q.to(BF16)
    try:
        fa.fa_set_max_ctas(ctas)
        got = fa.cache_attention(q.to(DEV), to_gpu(fa, (k, v, ks, vs)), i32(table), i32([L]))
        synced(fa)
    finally:
        fa.fa_set_max_ctas(0)
    floor = least_weight(n * Hq) * 2.0 ** -7 * v.float().abs().sum((0, 1, 2)).double().numpy()
    check_small_weights(q, got, R.Cache(k, v, ks, vs), table, [L], floor)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("n", [1, 5, 64])
def test_an_outlier_block_hides_nothing_in_columns_where_it_is_zero(fa, n, ctas):
    """A token with 90% of the weight in a block whose values have a scale 2^10 times the others', zero in half of the
    columns: there the output is made of the other tokens alone."""
    g = torch.Generator().manual_seed(n)
    page, D, Hq, H, L = 16, 128, 4, 1, 8192
    table, P, _ = R.make_table(g, [L], page)
    k, v, ks, vs = R.make_pools(g, P, H, page, D, E4M3)
    ks.fill_(1.0)
    vs.fill_(2.0 ** -7)
    k = (torch.randn(P, H, page, D, generator=g) * 0.25).to(E4M3)
    k.view(torch.uint8)[..., 0] = 0
    big = table[0][0]
    vs[big] = 2.0 ** 3
    k[big, 0, 3] = torch.zeros(D).to(E4M3)
    k[big, 0, 3, 0] = torch.tensor(16.0).to(E4M3)
    v.view(torch.uint8)[big] = 0
    v[big, 0, 3, D // 2:] = torch.full((D // 2,), 448.0).to(E4M3)
    q = torch.randn(1, Hq, n, D, generator=g) * 0.5
    q[..., 0] = 8.0
    q = q.to(BF16)
    try:
        fa.fa_set_max_ctas(ctas)
        got = fa.cache_attention(q.to(DEV), to_gpu(fa, (k, v, ks, vs)), i32(table), i32([L]))
        synced(fa)
    finally:
        fa.fa_set_max_ctas(0)
    floor = least_weight(n * Hq) * 2.0 ** 3 * v.float().abs().sum((0, 1, 2)).double().numpy()
    check_small_weights(q, got, R.Cache(k, v, ks, vs), table, [L], floor)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("track", [False, True])
@pytest.mark.parametrize("where", ["query", "key", "infinity"])
@pytest.mark.parametrize("n,D,page,lens", [(1, 128, 64, [700, 40]), (5, 64, 16, [9, 300]), (6, 256, 64, [900, 33]),
                                           (150, 128, 64, [150, 700]), (150, 64, 16, [400, 200])])
def test_not_a_number_is_told(fa, n, D, page, lens, where, track, ctas):
    """A row that sees a NaN score, or an infinite one, is NaN, its L too, and so is the weight of each token that it
    sees; the other rows, and the tokens that no such row sees, are as if nothing was wrong."""
    g = torch.Generator().manual_seed(n + D)
    B, Hq, H = len(lens), 4, 2
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, H, page, D, E4M3)
    q = torch.randn(B, Hq, n, D, generator=g).to(F16 if where == "infinity" else BF16)
    bad = np.zeros((B, Hq, n), bool)
    at = lens[0] - 1 - n // 2  # a token that the later half of sequence 0's rows sees
    qd = q.clone()
    raw = [t.clone() for t in pools]
    if where == "key":
        raw[0].view(torch.uint8)[table[0][at // page], 1, at % page, 5] = 0x7F
        bad[0, 2:] = lens[0] - n + np.arange(n) >= at
    else:
        bad[0, 1, n - 1] = bad[1, 3, 0] = True
        qd[0, 1, n - 1, 7] = qd[1, 3, 0, 7] = float("nan" if where == "query" else "inf")
        for b, h, i in ((0, 0, n - 1), (1, 1, 0)):  # (an infinite entry makes some score NaN or +inf)
            blocks = [x for x in table[b] if x >= 0]
            col = raw[0].float()[blocks, h // 2, :, 7].reshape(-1)[:lens[b] - n + i + 1]
            assert (col >= 0).any()
    w = w0 = None
    if track:
        w0 = torch.rand(B, H, max(lens), generator=g)
        w = w0.to(DEV)
    try:
        fa.fa_set_max_ctas(ctas)
        o, lse = fa.cache_attention(qd.to(DEV), to_gpu(fa, raw), i32(table), i32(lens), weights=w)
        synced(fa)
    finally:
        fa.fa_set_max_ctas(0)
    ref = R.Cache(*pools)
    ro, rl, rw, _, _ = R.attention(ref, q, table, lens)
    o, lse, there = o.cpu(), lse.cpu(), torch.from_numpy(bad)
    assert torch.isnan(o[there]).all() and torch.isnan(lse[there]).all()
    o[there], lse[there] = torch.from_numpy(ro)[there].to(o.dtype), torch.from_numpy(rl)[there].float()
    if track:
        w = w.cpu()
        for b in range(B):
            for h in range(H):
                rows = np.nonzero(bad[b, 2 * h:2 * h + 2].any(0))[0]
                seen = lens[b] - n + int(rows.max()) + 1 if len(rows) else 0
                assert torch.isnan(w[b, h, :seen]).all()
                w[b, h, :seen] = w0[b, h, :seen] + torch.from_numpy(rw)[b, h, :seen].float()
    check_attention(fa, ref, q, table, lens, (o, lse), w, w0)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("n,D", [(6, 64), (6, 256), (40, 128), (150, 64)])
def test_rows_that_see_nothing_are_zero_beside_a_nan_value(fa, n, D, ctas):
    """More rows than tokens, and padding behind n_q, in one row group with rows that see a NaN value."""
    g = torch.Generator().manual_seed(n)
    page, lens, n_q = 16, [n - 2, 60], [n, 3]
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, 2, page, D, E4M3)
    for b in range(2):
        pools[1].view(torch.uint8)[table[b][0], :, 0] = 0x7F
    q = torch.randn(2, 4, n, D, generator=g).to(BF16)
    try:
        fa.fa_set_max_ctas(ctas)
        o, lse = fa.cache_attention(q.to(DEV), to_gpu(fa, pools), i32(table), i32(lens), n_q=i32(n_q))
        synced(fa)
    finally:
        fa.fa_set_max_ctas(0)
    assert (o[0, :, :2] == 0).all() and torch.isneginf(lse[0, :, :2]).all()
    assert (o[1, :, 3:] == 0).all() and torch.isneginf(lse[1, :, 3:]).all()
    assert torch.isnan(o[0, :, 2:]).all() and torch.isfinite(lse[0, :, 2:]).all()
    assert torch.isnan(o[1, :, :3]).all() and torch.isfinite(lse[1, :, :3]).all()


@pytest.mark.parametrize("into", [True, False])
@pytest.mark.parametrize("L", [20, 5000, 50000])
@pytest.mark.parametrize("order", ["slots", "turned"])
def test_evict_keeps_the_latest_before_infinite_weights(fa, into, L, order):
    """Tokens pinned by an infinite weight, more of them than there is room beside the latest: the latest stay, then
    the pinned ones of the lowest slots; with room for all pins, all stay."""
    page, D, keep, recent, pins = 16, 64, 6, 3, 8
    inf = float("inf")
    M, extra = -(-L // page), 1
    cache = fa.kv_cache(M + extra, 1, D, page=page)
    w = torch.rand(1, 1, M * page, generator=torch.Generator().manual_seed(L))
    p = torch.arange(M * page, dtype=torch.int32)
    if order == "turned":  # the latest positions in the lowest slots
        p = (L - 1 - p).contiguous()
    p = p.view(1, 1, -1)
    latest = list(range(3)) if order == "turned" else list(range(L - 3, L))
    pinned = list(range(4, 4 + pins))
    w[0, 0, pinned] = inf
    w[0, 0, latest] = -inf  # (their weight does not count)
    wd, pd = w.to(DEV), p.to(DEV)
    table = i32([list(range(M))])
    kept = sorted(latest + pinned[:keep - recent])
    if into:
        wo, po = torch.zeros(1, 1, keep, device=DEV), torch.zeros(1, 1, keep, dtype=torch.int32, device=DEV)
        fa.cache_evict(cache, table, i32([L]), wd, pd, keep=keep, recent=recent, into=i32([[M]]), weights_out=wo, positions_out=po)
    else:
        fa.cache_evict(cache, table, i32([L]), wd, pd, keep=keep, recent=recent)
        wo, po = wd[:, :, :keep], pd[:, :, :keep]
    synced(fa)
    assert sorted(po[0, 0].tolist()) == sorted(p[0, 0, kept].tolist())
    assert sorted(wo[0, 0].tolist()) == sorted(w[0, 0, kept].tolist())


def test_status_tells_of_a_bad_index_behind_a_timeout(fa):
    """Both since the last call: one is reported, and the other by the next call."""
    cache = fa.kv_cache(2, 1, 64, page=16)
    x = torch.ones(1, 1, 1, 64, dtype=BF16, device=DEV)
    q = torch.randn(1, 4, 640, 128, device=DEV).to(BF16)
    try:
        fa.fa_set_timeout_cycles(1)
        fa.cache_append(cache, x, x, i32([[99]]), i32([0]))
        fa.attention(q, q, q, causal=True)
        first = fa.fa_sync_status(None)
    finally:
        fa.fa_set_timeout_cycles(0)
    assert first == fa.fa.FA_ERR_DEVICE_TIMEOUT
    assert fa.fa_sync_status(None) == fa.fa.FA_ERR_INVALID_ARGUMENT and "out of range" in fa.fa_last_error()
    assert fa.fa_sync_status(None) == fa.fa.FA_OK


@pytest.mark.parametrize("D,page,n,lens", [(256, 64, 1, [9000, 4000]), (128, 64, 5, [9000, 4000]), (256, 32, 2, [30000])])
def test_two_producers_unwind_at_once(fa, D, page, n, lens):
    """Two producers that stop at different tiles: neither waits for copies that the other never issues."""
    g = torch.Generator().manual_seed(D)
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, 2, page, D, E4M3)
    q = torch.randn(len(lens), 8, n, D, generator=g).to(BF16)
    cache, qd, t, ln = to_gpu(fa, pools), q.to(DEV), i32(table), i32(lens)
    fa.cache_attention(qd, cache, t, ln)
    torch.cuda.synchronize()
    longest, told = 0.0, 0
    try:
        for ctas in (0, 1, 8):
            fa.fa_set_max_ctas(ctas)
            for cycles in list(range(1, 4000, 100)) * 3:
                fa.fa_set_timeout_cycles(cycles)
                begin = time.monotonic()
                fa.cache_attention(qd, cache, t, ln)
                told += fa.fa_sync_status(None) == fa.fa.FA_ERR_DEVICE_TIMEOUT
                longest = max(longest, time.monotonic() - begin)
    finally:
        fa.fa_set_timeout_cycles(0)
        fa.fa_set_max_ctas(0)
    assert told > 0 and longest < 1.0, f"{told} expired, the longest took {longest:.2f} s"
    got = fa.cache_attention(qd, cache, t, ln)
    synced(fa)
    check_attention(fa, R.Cache(*pools), q, table, lens, got)
