"""GPU parity of decoding with drafts with its definition in 64 bits (tests/draft_reference.py)."""
import random

import numpy as np
import pytest
import torch

import cache_reference as R
import draft_reference as T

pytestmark = pytest.mark.gpu
E4M3, I8, BF16, F16, F32 = R.E4M3, R.I8, torch.bfloat16, torch.float16, torch.float32
DEV = "cuda:0"
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11}  # half a step, relative
SHAPES = ("chain", "star", "forest", "beam")


@pytest.fixture(scope="module")
def fa():
    import attention_forward_08_gb300 as fa
    assert fa.fa_sync_status(None) == 0
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def to_gpu(fa, pools):
    return fa.KVCache(*(t.to(DEV) for t in pools))


def synced(fa):
    assert fa.fa_sync_status(None) == 0, fa.fa_last_error()


def told(fa):
    assert fa.fa_sync_status(None) == fa.fa.FA_ERR_INVALID_ARGUMENT and "out of range" in fa.fa_last_error()
    assert fa.fa_sync_status(None) == 0


# ----------------------------------------------------------------- attention

def check_attention(ref, q, table, lens, trees, got, got_w=None, w0=None, **kw):
    """L: fp32 sums of D products, 2^-18 of the largest sum of |q k| (D = 256 steps of 2^-24 at worst, 2^-16, of
    which roundings to nearest reach a quarter at most here), and 1e-6 for the logarithm.  O: half a step of the
    output, and of the weights' f16 form (2^-11) and twice L's error times sum of p |v|.  Weights: L's error twice, and
    2^-22 for the additions."""
    o, lse = (t.double().cpu().numpy() for t in got)
    ro, rl, rw, a, sabs = T.attention(ref, q, table, lens, trees, **kw)
    tol_l = (2.0 ** -18 * sabs + 1e-6)[:, None, None]
    empty = np.isneginf(rl)
    np.testing.assert_array_equal(np.isneginf(lse), empty)
    assert np.all(o[empty] == 0.0)
    assert np.all(np.isfinite(o))
    d = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, rl))
    assert np.all(d <= tol_l), f"max |dL| {d.max():.3e} at {np.unravel_index(d.argmax(), d.shape)}, allowed {tol_l.max():.3e}"
    tol_o = HALF[q.dtype] * np.abs(ro) + (HALF[F16] + 2 * tol_l[..., None]) * a + 1e-7
    d = np.abs(o - ro)
    assert np.all(d <= tol_o), f"max |dO| {d.max():.3e} at {np.unravel_index(d.argmax(), d.shape)}, {(d / tol_o).max():.2f} of the tolerance"
    if got_w is not None:
        w = got_w.double().cpu().numpy()
        want = w0.double().cpu().numpy().copy()
        want[:, :, :rw.shape[2]] += rw
        tol = 2.0 ** -22 * np.abs(want)
        tol[:, :, :rw.shape[2]] += 2 * tol_l * rw
        d = np.abs(w - want)
        assert np.all(d <= tol), f"max |dw| {d.max():.3e} at {np.unravel_index(d.argmax(), d.shape)}"


def tree_case(fa, *, kind=E4M3, io=BF16, D=128, page=64, Hq=4, Hkv=2, lens=(100,), n=5, n_q=None, shape="beam",
              shared=False, track=False, seed=0, **kw):
    g = torch.Generator().manual_seed(seed + D + page + sum(lens) + n)
    rng = random.Random(seed + n)
    lens, B = list(lens), len(lens)
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, Hkv, page, D, kind)
    ref = R.Cache(*pools)
    for t in pools[:2]:
        R.spoil(t, table, lens, page)
    q = torch.randn(B, Hq, n, D, generator=g).to(io)
    trees = [T.random_tree(rng, n, SHAPES[(b + seed) % 4] if shape == "all" else shape) for b in range(B)]
    if shared:
        trees = trees[:1] * B
    given = [list(t) for t in trees]
    for t, rows in zip(given, n_q or []):  # rows that are none: never read
        t[rows:] = [10 ** 6] * (n - rows)
    cache = to_gpu(fa, pools)
    w = w0 = None
    if track:
        w0 = torch.rand(B, Hkv, max(1, max(lens)) + 3, generator=g)
        w = w0.to(DEV)
    got = fa.cache_attention(q.to(DEV), cache, i32(table), i32(lens), n_q=None if n_q is None else i32(list(n_q)),
                             weights=w, tree=i32(given[0] if shared else given), **kw)
    synced(fa)
    check_attention(ref, q, table, lens, trees, got, w, w0, n_q=n_q, **kw)
    return got


@pytest.mark.parametrize("kind", [E4M3, I8])
@pytest.mark.parametrize("io", [BF16, F16])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128), (128, 16), (256, 32)])
@pytest.mark.parametrize("n", [1, 5, 16, 40])
def test_tree(fa, kind, io, D, page, n):
    """Contexts of no token, and around a block's and a tile's end, trees of every shape."""
    tree_case(fa, kind=kind, io=io, D=D, page=page, Hq=8, Hkv=2, n=n, shape="all",
              lens=(n, n + 1, n + 31, n + 63, n + 64, n + 127, 700), track=page == 64)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (32, 8), (16, 1), (24, 1), (64, 2), (130, 1)])
@pytest.mark.parametrize("n", [2, 9])
def test_tree_groups(fa, Hq, Hkv, n):
    tree_case(fa, Hq=Hq, Hkv=Hkv, n=n, lens=(700, 33, 256), track=True)


@pytest.mark.parametrize("n", [8, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D,page,kind,io,Hq,Hkv", [(128, 64, E4M3, BF16, 2, 2), (64, 16, I8, F16, 3, 1),
                                                   (256, 128, E4M3, F16, 2, 1)])
def test_tree_sizes(fa, n, shape, D, page, kind, io, Hq, Hkv):
    tree_case(fa, kind=kind, io=io, D=D, page=page, Hq=Hq, Hkv=Hkv, n=n, shape=shape, lens=(n, n + 77, 640),
              track=n in (33, 129))


@pytest.mark.parametrize("n", [1, 6, 30, 100])
@pytest.mark.parametrize("window", [1, 2, 5, 64, 100, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("shape", ["chain", "beam", "forest"])
def test_tree_window(fa, n, window, shape):
    """A window that ends among the drafts above, at their begin, before them; as the positions say, not the slots."""
    tree_case(fa, n=n, lens=(n, 3 + n, 130 + n, 777), window=window, shape=shape, track=window in (2, 100))


@pytest.mark.parametrize("n", [3, 20, 70])
@pytest.mark.parametrize("softcap,scale", [(0.5, None), (20.0, None), (0.0, -0.1), (0.0, 0.0), (0.0, 1.0), (30.0, 0.5)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_softcap_and_scale(fa, n, softcap, scale, D):
    tree_case(fa, n=n, D=D, lens=(n + 200, 400), softcap=softcap, scale=scale, window=0 if D == 64 else 90, track=D == 64)


@pytest.mark.parametrize("n,lens,n_q", [
    (4, (0, 2, 9, 4), None),                 # more drafts than tokens: the first are not there
    (6, (100, 100, 7, 0, 3), (6, 2, 0, 0, 3)),
    (90, (300, 300, 0, 130, 40), (90, 1, 0, 90, 40)),
    (90, (100, 0, 89, 50), None),
])
@pytest.mark.parametrize("shape", ["chain", "beam", "star"])
def test_tree_empty_rows_and_padding(fa, n, lens, n_q, shape):
    tree_case(fa, n=n, lens=lens, n_q=n_q, shape=shape, track=True)
    tree_case(fa, n=n, lens=lens, n_q=n_q, shape=shape, D=64, page=16, kind=I8, window=20, track=True)


@pytest.mark.parametrize("n", [4, 50])
def test_tree_shared(fa, n):
    tree_case(fa, n=n, lens=(n + 5, 300, 90, n), shared=True)


def test_tree_largest(fa):
    tree_case(fa, n=1024, lens=(1500, 1024), Hq=1, Hkv=1, D=64, shape="chain")
    tree_case(fa, n=1000, lens=(1100,), Hq=2, Hkv=1, D=128, shape="beam", window=70, track=True)


@pytest.mark.parametrize("n", [7, 40])
def test_tree_long_cache(fa, n):
    tree_case(fa, n=n, lens=(70001,), Hq=4, Hkv=1, track=True)
    tree_case(fa, n=n, lens=(9000, 12345, 40), Hq=8, Hkv=8, page=16)


@pytest.mark.parametrize("ctas", [1, 2, 7])
@pytest.mark.parametrize("kind,io,D,page,Hq,Hkv,n", [
    (E4M3, BF16, 128, 64, 8, 2, 3), (I8, F16, 64, 16, 6, 3, 9), (E4M3, F16, 256, 128, 4, 2, 5), (E4M3, BF16, 128, 16, 8, 2, 20),
    (I8, BF16, 64, 32, 8, 1, 40), (I8, BF16, 256, 16, 8, 1, 9),
])
def test_tree_long_parts(fa, ctas, kind, io, D, page, Hq, Hkv, n):
    """Few thread blocks: each goes round its ring many times, over parts of several sequences and heads."""
    fa.fa_set_max_ctas(ctas)
    try:
        tree_case(fa, kind=kind, io=io, D=D, page=page, Hq=Hq, Hkv=Hkv, n=n, lens=(2500, n, 777, 0, 1300), track=True)
        tree_case(fa, kind=kind, io=io, D=D, page=page, Hq=Hq, Hkv=Hkv, n=n, lens=(4000,) * 3, window=900)
    finally:
        fa.fa_set_max_ctas(0)


@pytest.mark.parametrize("n", [1, 5, 25, 150])
def test_chain_is_plain_attention(fa, n):
    """The same rows with and without their chain as a tree."""
    g = torch.Generator().manual_seed(n)
    page, D, lens = 32, 128, [n + 60, n + 3]
    table, P, _ = R.make_table(g, lens, page)
    cache = to_gpu(fa, R.make_pools(g, P, 2, page, D, E4M3))
    q = torch.randn(2, 8, n, D, generator=g).to(BF16).to(DEV)
    chain = i32([i - 1 for i in range(n)])
    a = fa.cache_attention(q, cache, i32(table), i32(lens), window=50)
    b = fa.cache_attention(q, cache, i32(table), i32(lens), window=50, tree=chain)
    synced(fa)
    # each is within half a step of O and 2^-11 of weights in [0, 1] of what both compute; L as in check_attention
    scale = a[0].double().abs().max().item()
    assert (a[0].double() - b[0].double()).abs().max().item() <= 2 * (HALF[BF16] + 2 * HALF[F16]) * 4 * scale
    torch.testing.assert_close(a[1], b[1], rtol=0, atol=1e-4)


@pytest.mark.parametrize("n", [4, 40])
def test_tree_strided(fa, n):
    """Token-major q and output, a tree and a table that are slices of wider ones, pools interleaved."""
    g = torch.Generator().manual_seed(n)
    P, H, page, D, lens = 16, 2, 32, 128, [n + 60, n + 3]
    raw = torch.zeros(P, page, 2, H, D, dtype=torch.uint8, device=DEV)
    pools = R.make_pools(g, P, H, page, D, I8)
    views = [raw[:, :, i].permute(0, 2, 1, 3).view(I8) for i in range(2)]
    for a, b in zip(views, pools):
        a.copy_(b)
    cache, ref = fa.KVCache(*views, pools[2].to(DEV), pools[3].to(DEV)), R.Cache(*pools)
    table = [[5, 0, 7, 2], [1, 3, 4, 6]]
    wide = torch.full((2, 9), -1, dtype=torch.int32, device=DEV)
    wide[:, 4:8] = i32(table)
    trees = [T.random_tree(random.Random(b), n, "beam") for b in range(2)]
    tree = torch.full((2, n + 3), 77, dtype=torch.int32, device=DEV)
    tree[:, 2:2 + n] = i32(trees)
    q = torch.randn(2, n, 6, D, generator=g).to(F16)
    out = torch.full((2, n, 6, D), float("nan"), dtype=F16, device=DEV)
    o, lse = fa.cache_attention(q.to(DEV).transpose(1, 2), cache, wide[:, 4:8], i32(lens), out=out.transpose(1, 2),
                                tree=tree[:, 2:2 + n])
    synced(fa)
    assert o.data_ptr() == out.data_ptr()
    check_attention(ref, q.transpose(1, 2), table, lens, trees, (o, lse))


@pytest.mark.parametrize("n", [5, 50])
def test_tree_bad_entries(fa, n):
    """A parent that is no earlier row counts as none; a bad table entry hides its tokens; both are told."""
    g = torch.Generator().manual_seed(3)
    table, P, _ = R.make_table(g, [160, 160], 16)
    pools = R.make_pools(g, P, 1, 16, 64, E4M3)
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    q = torch.randn(2, 2, n, 64, generator=g).to(BF16)
    trees = [[-1, 0, 2, 99, 3] + [4] * (n - 5), [-1, -7, 1, 0, -2 ** 31] + [4] * (n - 5)]
    o, lse = fa.cache_attention(q.to(DEV), cache, i32(table), i32([160, 160]), tree=i32(trees))
    told(fa)
    check_attention(ref, q, table, [160, 160], trees, (o, lse))
    bad = [list(r) for r in table]
    bad[0][0], bad[1][0] = P, -5
    good = [T.random_tree(random.Random(1), n, "beam")] * 2
    o, lse = fa.cache_attention(q.to(DEV), cache, i32(bad), i32([160, 160]), tree=i32(good))
    told(fa)
    check_attention(ref, q, table, [160, 160], good, (o, lse), hidden=range(16))
    # outside the window it is not needed
    o, lse = fa.cache_attention(q.to(DEV), cache, i32(bad), i32([160, 160]), tree=i32(good), window=140 - n)
    synced(fa)
    check_attention(ref, q, table, [160, 160], good, (o, lse), window=140 - n)


@pytest.mark.parametrize("n", [6, 20, 60])
def test_tree_nan_and_infinite_scores(fa, n):
    """A NaN key makes the rows that see it NaN, and their weights; a sibling's row stays what it is."""
    g = torch.Generator().manual_seed(6)
    L, page, D = 100 + n, 16, 64
    table, P, _ = R.make_table(g, [L], page)
    pools = R.make_pools(g, P, 1, page, D, E4M3)
    tree = [-1, 0, 0, 2, 1, 2] + [4] * (n - 6)
    slot = 100 + 2  # node 2's key
    pools[0].view(torch.uint8)[table[0][slot // page], 0, slot % page] = 0x7F
    cache = to_gpu(fa, pools)
    q = torch.randn(1, 2, n, D, generator=g).to(BF16)
    w = torch.zeros(1, 1, L, device=DEV)
    o, lse = fa.cache_attention(q.to(DEV), cache, i32(table), i32([L]), tree=i32([tree]), weights=w)
    synced(fa)
    sees = torch.tensor([2 in T.line(tree, i) for i in range(n)])
    assert torch.equal(torch.isnan(lse[0, 0].cpu()), sees) and torch.equal(torch.isnan(o[0, 1]).all(-1).cpu(), sees)
    hidden = torch.tensor([i for i in range(n) if not any(i in T.line(tree, k) for k in (2, 3, 5))])
    assert not torch.isnan(w[0, 0, 100 + hidden.to(DEV)]).any() and torch.isnan(w[0, 0, :100]).all()


@pytest.mark.parametrize("D,page,kind,io,Hq,Hkv,n", [
    (64, 16, E4M3, BF16, 2, 1, 6), (128, 64, I8, F16, 4, 2, 8), (128, 16, E4M3, BF16, 8, 2, 6), (64, 16, I8, F16, 2, 1, 20),
    (128, 64, E4M3, BF16, 2, 1, 60), (256, 16, E4M3, F16, 2, 1, 9), (256, 64, I8, BF16, 4, 2, 40), (64, 32, E4M3, F16, 8, 4, 90)])
@pytest.mark.parametrize("L", [0, 100, 900])
@pytest.mark.parametrize("ctas", [0, 2])
@pytest.mark.parametrize("track", [False, True])
def test_tree_infinite_scores(fa, D, page, kind, io, Hq, Hkv, n, L, ctas, track):
    """Node 2's key has a score of +infinity with the rows of a group's first head, all others -infinity: what sees it
    is NaN, and the weights of the tokens that it sees; the head's other rows see as good as nothing, and the other
    heads' are what they are."""
    g = torch.Generator().manual_seed(n + L)
    group, length = Hq // Hkv, L + n
    table, P, _ = R.make_table(g, [length], page)
    pools = R.make_pools(g, P, Hkv, page, D, kind)
    tree = [-1, 0, 0, 2, 1, 2] + [4] * (n - 6)
    pools[0][..., 0] = torch.tensor(-8.0).to(kind)
    pools[0][table[0][(L + 2) // page], :, (L + 2) % page, 0] = torch.tensor(8.0).to(kind)
    q = torch.randn(1, Hq, n, D, generator=g).to(io)
    plain = q.clone()
    q[:, ::group, :, 0] = float("inf")
    w = torch.zeros(1, Hkv, length, device=DEV)
    fa.fa_set_max_ctas(ctas)
    try:
        o, lse = fa.cache_attention(q.to(DEV), to_gpu(fa, pools), i32(table), i32([length]), tree=i32([tree]),
                                    weights=w if track else None)
    finally:
        fa.fa_set_max_ctas(0)
    synced(fa)
    o, lse, w = o.double().cpu(), lse.double().cpu(), w.double().cpu()
    sees = torch.tensor([2 in T.line(tree, i) for i in range(n)])
    assert torch.isnan(lse[:, ::group, sees]).all() and torch.isnan(o[:, ::group, sees]).all()
    assert torch.isneginf(lse[:, ::group, ~sees]).all() and (o[:, ::group, ~sees] == 0).all()
    others = torch.arange(Hq) % group > 0
    for h in range(Hkv):  # (each group's other heads, by themselves)
        part = R.Cache(*(t[:, h:h + 1] for t in pools))
        mine = others.clone()
        mine[:h * group], mine[(h + 1) * group:] = False, False
        ro, rl, rw, a, sabs = T.attention(part, plain[:, mine], table, [length], [tree])
        tol_l = 2.0 ** -18 * sabs[0] + 1e-6  # (as in check_attention)
        assert np.all(np.abs(lse[:, mine].numpy() - rl) <= tol_l)
        assert np.all(np.abs(o[:, mine].numpy() - ro) <= HALF[io] * np.abs(ro) + (HALF[F16] + 2 * tol_l) * a + 1e-7)
        if track:
            seen = T.visible(tree, length, n)[sees.numpy()].any(0)
            hidden = np.nonzero(~seen)[0]
            assert 0 < len(hidden) < n and torch.isnan(w[0, h][torch.from_numpy(seen)]).all()
            assert np.all(np.abs(w[0, h, hidden].numpy() - rw[0, 0, hidden]) <= (2.0 ** -22 + 2 * tol_l) * rw[0, 0, hidden])


def many_rows(fa, D, page, Hq, Hkv, n, lens, kind=E4M3):
    g = torch.Generator().manual_seed(D + n)
    rng = random.Random(n)
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, Hkv, page, D, kind)
    q = torch.randn(len(lens), Hq, n, D, generator=g).to(BF16)
    trees = [T.random_tree(rng, n, SHAPES[b % 4]) for b in range(len(lens))]
    cache, args = to_gpu(fa, pools), (i32(table), i32(lens))
    qd, tree = q.to(DEV), i32(trees)
    return (lambda: fa.cache_attention(qd, cache, *args, tree=tree)), (R.Cache(*pools), q, table, lens, trees)


# (rows four times, twice and once in a tile, two row groups, and heads of 256; the decode kernel's two tiles)
MANY_ROWS = [(128, 64, 8, 2, 5, [700, 300]), (64, 16, 8, 2, 12, [900, 201]), (128, 16, 4, 1, 30, [1000]),
             (128, 64, 8, 1, 30, [400, 2000]), (256, 64, 8, 2, 9, [400, 90]), (128, 64, 4, 2, 2, [300, 40])]


@pytest.mark.parametrize("ctas", [0, 3, 40])
@pytest.mark.parametrize("n,kw", [(12, {}), (40, dict(D=64, page=16, kind=I8)), (70, dict(track=True)),
                                  (10, dict(D=256, window=90, track=True))])
def test_tree_many_sequences(fa, n, kw, ctas):
    """More sequences than a warp has lanes, most of them short: thread blocks with many segments, with a few keys, with
    none; sequences without drafts and without tokens between them."""
    lens = [(37 * b) % 300 + n if b % 5 else (b % 3) * n for b in range(75)]
    n_q = [min(length, n if b % 4 else b % (n + 1)) for b, length in enumerate(lens)]
    lens[40] = 9000
    try:
        fa.fa_set_max_ctas(ctas)
        tree_case(fa, n=n, lens=lens, n_q=n_q, shape="all", **kw)
    finally:
        fa.fa_set_max_ctas(0)


@pytest.mark.parametrize("n", [33, 130])
@pytest.mark.parametrize("window", [1, 3, 40, 200])
@pytest.mark.parametrize("D,page", [(64, 16), (256, 64)])
def test_tree_weights_with_a_window(fa, n, window, D, page):
    """Windows that end in a line of drafts, at their begin and before them, and what the tokens there got."""
    tree_case(fa, n=n, D=D, page=page, Hq=2, Hkv=1, lens=(n, n + 1, n + 31, n + 32, n + 300), window=window, shape="all",
              track=True, softcap=5.0 if window == 3 else 0.0)


@pytest.mark.parametrize("D,page,Hq,Hkv,n,width", [
    (64, 16, 2, 1, 5, 0), (64, 16, 2, 1, 16, 0), (64, 16, 2, 1, 17, 0), (64, 16, 2, 1, 60, 0), (64, 16, 1, 1, 130, 0),
    (128, 16, 8, 2, 8, 0), (128, 16, 8, 2, 9, 0), (128, 64, 8, 2, 20, 0), (128, 32, 8, 2, 6, 1 << 20),
    (256, 16, 2, 1, 8, 0), (256, 16, 2, 1, 9, 0), (256, 32, 4, 2, 40, 0), (256, 128, 4, 1, 3, 1 << 20)])
@pytest.mark.parametrize("window", [3, 100])
def test_tree_weights_need_no_blocks_behind_the_window(fa, D, page, Hq, Hkv, n, width, window):
    """Table entries of tokens that a window hides from every draft may be anything, with scores that are kept and
    without; the window begins at every place of 32 tokens."""
    g = torch.Generator().manual_seed(n + D)
    lens = [n + 160 + 7 * b for b in range(33)]
    table, P, _ = R.make_table(g, lens, page, width=max(width // page, -(-max(lens) // page)))
    pools = R.make_pools(g, P, Hkv, page, D, E4M3)
    gone = [[P + 7 if (m + 1) * page <= length - n - window + 1 else x for m, x in enumerate(r)] for r, length in zip(table, lens)]
    assert any(P + 7 in r for r in gone)
    q = torch.randn(len(lens), Hq, n, D, generator=g).to(BF16)
    trees = [T.random_tree(random.Random(b), n, SHAPES[b % 4]) for b in range(len(lens))]
    w0 = torch.rand(len(lens), Hkv, max(lens) + 3, generator=g)
    w = w0.to(DEV)
    got = fa.cache_attention(q.to(DEV), to_gpu(fa, pools), i32(gone), i32(lens), tree=i32(trees), weights=w, window=window)
    synced(fa)
    check_attention(R.Cache(*pools), q, table, lens, trees, got, w, w0, window=window)


@pytest.mark.parametrize("ctas", [0, 1])
@pytest.mark.parametrize("cycles", [1, 300, 3000, 30000])
@pytest.mark.parametrize("D,page,Hq,Hkv,n,lens", MANY_ROWS)
def test_tree_wait_bounds_then_the_next_call_is_right(fa, D, page, Hq, Hkv, n, lens, cycles, ctas):
    """Copies, products and stores that are under way when a wait expires are done before the block gives back its
    memory."""
    call, ref = many_rows(fa, D, page, Hq, Hkv, n, lens)
    torch.cuda.synchronize()
    try:
        fa.fa_set_max_ctas(ctas)
        for _ in range(3):
            fa.fa_set_timeout_cycles(cycles)
            call()
            fa.fa_set_timeout_cycles(0)
            got = call()
            assert fa.fa_sync_status(None) in (fa.fa.FA_OK, fa.fa.FA_ERR_DEVICE_TIMEOUT), fa.fa_last_error()
            check_attention(*ref, got)
    finally:
        fa.fa_set_timeout_cycles(0)
        fa.fa_set_max_ctas(0)


@pytest.mark.parametrize("D,page,Hq,Hkv,n,lens", MANY_ROWS + [
    (128, 64, 32, 8, 16, [5000 - 300 * b for b in range(16)]), (64, 16, 32, 32, 33, [900 + 7 * b for b in range(5)]),
    (256, 16, 16, 2, 13, [3000 - 431 * b for b in range(7)]), (128, 64, 8, 1, 104, [9000])])
def test_tree_results_do_not_change_from_run_to_run(fa, D, page, Hq, Hkv, n, lens):
    call, ref = many_rows(fa, D, page, Hq, Hkv, n, lens)
    o, lse = call()
    check_attention(*ref, (o, lse))
    for _ in range(6):
        again = call()
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    synced(fa)


# ----------------------------------------------------------------- verification

def verify_case(fa, *, n=6, V=1000, B=3, dtype=F32, drawn=True, shape="beam", seed=0, sharp=2.0, n_q=None, u=None,
                u_next=None, change=None, pad=0):
    """Against the definition in 64 bits: whole numbers, so equal.  (Two ways of summing differ by 2^-48 of the sums;
    none of these random numbers lies that near a border.)"""
    g = torch.Generator().manual_seed(seed + n * 7 + V)
    rng = random.Random(seed + n)
    trees = [T.random_tree(rng, n, shape) for _ in range(B)]
    z = torch.randn(B, n, V, generator=g) * sharp
    q = torch.softmax(z, -1)
    p = torch.softmax(z + 0.7 * torch.randn(B, n, V, generator=g), -1)
    tokens = torch.zeros(B, n, dtype=torch.int32)
    for b in range(B):
        for i in range(1, n):
            row = q[b, max(trees[b][i], 0)]
            if drawn:
                tokens[b, i] = torch.multinomial(row, 1, generator=g)
            else:
                rank = sum(trees[b][j] == trees[b][i] for j in range(i))
                tokens[b, i] = torch.topk(row, min(V, rank + 1)).indices[-1]
    p, q = p.to(dtype), q.to(dtype)
    u = torch.rand(B, n, generator=g) if u is None else u
    u_next = torch.rand(B, generator=g) if u_next is None else u_next
    if change is not None:
        change(p, q, tokens)
    pd = torch.empty(B, n, V + pad, dtype=dtype, device=DEV)[:, :, pad:].copy_(p)
    qd = torch.empty(B, n, V + 2 * pad, dtype=dtype, device=DEV)[:, :, pad:pad + V].copy_(q) if drawn else None
    got = fa.verify_drafts(pd, tokens.to(DEV), i32(trees), u.to(DEV), u_next.to(DEV), p_draft=qd,
                           n_q=None if n_q is None else i32(list(n_q)))
    path, count, token = (t.cpu().tolist() for t in got)
    for b in range(B):
        want, t = T.verify(p[b].double().numpy(), tokens[b].tolist(), trees[b], u[b].tolist(), u_next[b].item(),
                           q[b].double().numpy() if drawn else None, nodes=None if n_q is None else n_q[b])
        assert path[b] == want + [-1] * (n - len(want)) and count[b] == len(want) and token[b] == t, b
    return path, count, token


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4097, 50001])
@pytest.mark.parametrize("shape", SHAPES)
def test_verify(fa, drawn, dtype, V, shape):
    verify_case(fa, V=V, dtype=dtype, drawn=drawn, shape=shape, n=9 if V < 50000 else 5)
    synced(fa)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 100, 513, 1024])
@pytest.mark.parametrize("shape", ["star", "beam"])
def test_verify_tree_sizes(fa, drawn, n, shape):
    """Stars: many children are rejected in turn, each with a sum over what is left."""
    verify_case(fa, n=n, V=150, B=2, drawn=drawn, shape=shape, sharp=1.0)
    synced(fa)


def test_verify_largest_vocabulary(fa):
    for drawn in (True, False):
        verify_case(fa, n=3, V=1 << 20, B=1, drawn=drawn, shape="star", sharp=4.0)
    synced(fa)


@pytest.mark.parametrize("B", [20, 40, 80])
@pytest.mark.parametrize("n,V", [(2, 1 << 20), (7, 70001)])
def test_verify_large_vocabularies_of_many(fa, B, n, V):
    """The blocks of a sequence are as many as run at once, unless what is rejected has no room."""
    verify_case(fa, n=n, V=V if B < 80 else V // 2, B=B, dtype=BF16, drawn=False, shape="star", sharp=3.0)
    synced(fa)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_results_do_not_change_from_run_to_run(fa, drawn):
    got = [verify_case(fa, n=12, V=30011, B=24, drawn=drawn, seed=3) for _ in range(3)]
    assert got[0] == got[1] == got[2]
    synced(fa)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_many_sequences(fa, drawn):
    got = [verify_case(fa, n=6, V=301, B=200, drawn=drawn, seed=s)[1] for s in range(4)]
    assert len(set(sum(got, []))) > 2  # (paths of several lengths)
    synced(fa)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("u,u_next", [(0.0, 0.0), (0.0, 1 - 2.0 ** -24), (1 - 2.0 ** -24, 0.0), (1 - 2.0 ** -24, 1 - 2.0 ** -24)])
def test_verify_extreme_random_numbers(fa, drawn, u, u_next):
    """0: everything with a chance is accepted, the first token with any is next; the largest below 1."""
    verify_case(fa, n=12, V=77, B=4, drawn=drawn, u=torch.full((4, 12), u), u_next=torch.full((4,), u_next))
    synced(fa)


def test_verify_random_numbers_out_of_range(fa):
    """1 and more, negative, NaN: as 1, 0 and 0 for the next token; a test with NaN fails."""
    for x in (1.0, 5.0, -1.0, float("nan")):
        verify_case(fa, n=5, V=70, B=2, u=torch.full((2, 5), x), u_next=torch.full((2,), x))
    synced(fa)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_special_probabilities(fa, drawn):
    """Zeros (a cut distribution), one-hot rows, rows without any, NaN, negative and infinite entries."""
    def cut(p, q, tokens):
        p[p < 0.01] = 0.0

    def one_hot(p, q, tokens):
        p.zero_()
        p[..., 17] = 1.0
        tokens[:, ::2] = 17

    def none(p, q, tokens):
        p.zero_()

    def equal(p, q, tokens):
        q.copy_(p)

    def odd(p, q, tokens):
        p[..., 3], p[..., 5], p[..., 7] = float("nan"), -1.0, float("inf")
        q[..., 4], q[..., 6], q[..., 7] = float("nan"), -1.0, float("inf")
        tokens[:, 1] = 3

    for change in (cut, one_hot, none, equal, odd):
        for shape in ("star", "chain"):
            got = verify_case(fa, n=8, V=90, B=3, drawn=drawn, shape=shape, change=change)
            if change is one_hot:
                assert got[2] == [17] * 3
            if change is none:
                assert got[1] == [1] * 3 and got[2] == [0] * 3
    synced(fa)


def test_verify_same_candidate_twice(fa):
    def twice(p, q, tokens):
        tokens[:, 1:] = tokens[:, 1:2]

    verify_case(fa, n=6, V=50, B=8, drawn=False, shape="star", change=twice)
    verify_case(fa, n=6, V=50, B=8, drawn=True, shape="star", change=twice)
    synced(fa)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_verify_what_two_rejections_leave_is_not_rounded_away(fa, dtype):
    """Entry 0 of what two rejected drafts (of token 2, which the target never takes) leave is p - C q with a C of more
    than 24 bits: a difference in the last place of p, or 0; u_next 0 takes the first token that has any.  (The terms
    are fp32 numbers or less, so p - C q is off by 2^-46 of p at most with C in 48 bits; cases nearer to 0 are left out.)"""
    B, V = 4000, 3
    rng = np.random.default_rng(7)
    p, q = np.zeros((B, V)), np.zeros((B, V))
    f = lambda x: torch.tensor(x).to(dtype).double().numpy()
    q[:, 0], q[:, 1] = f(rng.uniform(0.1, 0.4, B)), f(rng.uniform(0.1, 0.3, B))
    q[:, 2] = f(1.0 - q[:, 0] - q[:, 1])
    p[:, 1] = f(np.maximum(1.0 - q[:, 0] * (1.0 + q[:, 2]), q[:, 1]))
    for _ in range(40):  # p[0] next to C q[0]
        z = np.maximum(p[:, 0] - q[:, 0], 0.0) + (p[:, 1] - q[:, 1])
        p[:, 0] = f((1.0 + z) * q[:, 0])
    z = np.maximum(p[:, 0] - q[:, 0], 0.0) + (p[:, 1] - q[:, 1])
    left = p[:, 0] - q[:, 0] - z * q[:, 0]
    use = np.abs(left) > 2.0 ** -40
    p, q, left = p[use], q[use], left[use]
    B = len(p)
    assert min((left > 0).mean(), (left < 0).mean()) > 0.1
    tokens, tree = i32([[0, 2, 2]] * B), i32([-1, 0, 0])
    dev = lambda x: torch.tensor(x).to(dtype).to(DEV)[:, None].expand(B, 3, V)
    path, count, token = fa.verify_drafts(dev(p), tokens, tree, torch.full((B, 3), 0.5, device=DEV),
                                          torch.zeros(B, device=DEV), p_draft=dev(q))
    synced(fa)
    assert (count == 1).all()
    want = [T.verify(np.tile(p[b], (3, 1)), [0, 2, 2], [-1, 0, 0], [0.5] * 3, 0.0, np.tile(q[b], (3, 1)))[1] for b in range(B)]
    assert np.array_equal(want, np.where(left > 0, 0, 1))
    wrong = np.nonzero(token.cpu().numpy() != want)[0]
    assert len(wrong) == 0, f"{len(wrong)} of {B}; the first, {wrong[0]}: {token[wrong[0]]} for {want[wrong[0]]}"


def test_verify_padding_and_strides(fa):
    verify_case(fa, n=7, V=333, B=5, n_q=(7, 0, 1, 3, 6), pad=3)
    verify_case(fa, n=7, V=333, B=5, n_q=(7, 0, 1, 3, 6), drawn=False, dtype=BF16, pad=1)
    synced(fa)


def test_verify_bad_entries(fa):
    """A token outside the vocabulary is rejected, a parent that is none is never reached, a count is cut; all told."""
    def tokens_out(p, q, tokens):
        tokens[:, 1] = 60
        tokens[:, 2] = -3

    for drawn in (True, False):
        verify_case(fa, n=6, V=50, B=2, drawn=drawn, shape="star", change=tokens_out)
        told(fa)
    p = torch.full((1, 4, 8), 0.125, device=DEV)
    u, x = torch.zeros(1, 4, device=DEV), torch.zeros(1, device=DEV)
    path, count, token = fa.verify_drafts(p, i32([[0, 1, 2, 3]]), i32([[-1, 0, 9, 2]]), u, x, n_q=i32([7]))
    told(fa)
    assert path.tolist() == [[0, 1, -1, -1]] and count.tolist() == [2] and token.tolist() == [0]


def test_verify_keeps_the_target_distribution(fa):
    """20,000 sequences with one tree's probabilities: the first token behind node 0 is distributed as p[0]: a chi-square
    statistic of 7 degrees of freedom is above 29.9 once in 10,000 tries."""
    B, n, V = 20000, 4, 8
    g = torch.Generator().manual_seed(12)
    q1, p1 = torch.softmax(torch.randn(n, V, generator=g), -1), torch.softmax(torch.randn(n, V, generator=g), -1)
    tokens = torch.multinomial(q1[0], B * n, replacement=True, generator=g).view(B, n).to(torch.int32)
    u, x = torch.rand(B, n, generator=g), torch.rand(B, generator=g)
    path, count, token = (t.cpu() for t in fa.verify_drafts(
        p1.to(DEV).expand(B, n, V), tokens.to(DEV), i32([-1, 0, 0, 0]), u.to(DEV), x.to(DEV),
        p_draft=q1.to(DEV).expand(B, n, V)))
    synced(fa)
    first = torch.where(count > 1, tokens.gather(1, path[:, 1:2].clamp_min(0).long())[:, 0], token)
    seen, want = torch.bincount(first.long(), minlength=V).double(), p1[0].double() * B
    assert ((seen - want) ** 2 / want).sum() < 29.9
    assert 0.3 < (count > 1).double().mean() < 0.999


# ----------------------------------------------------------------- acceptance

def accept_case(fa, *, kind=E4M3, D=64, page=16, H=2, lens=(100,), n=10, counts=(4,), n_q=None, seed=0, track=True, W=None,
                alias=False, paths=None):
    g = torch.Generator().manual_seed(seed + sum(lens) + n)
    rng = random.Random(seed + n)
    lens, B = list(lens), len(lens)
    n_q = [n] * B if n_q is None else list(n_q)
    table, P, _ = R.make_table(g, lens, page)
    pools = R.make_pools(g, P, H, page, D, kind)
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    if paths is None:
        paths = [sorted(rng.sample(range(rows), k)) for rows, k in zip(n_q, counts)]
    path = torch.full((B, n), -1, dtype=torch.int32)
    for b, line in enumerate(paths):
        path[b, :len(line)] = torch.tensor(line, dtype=torch.int32)
    W = len(table[0]) * page + 3 if W is None else W
    w = torch.rand(B, H, W, generator=g)
    want_w, wd = w.numpy().copy(), w.to(DEV)
    want = T.accept(ref, table, lens, paths, list(counts), n_q, want_w if track else None)
    ld = i32(lens)
    got = fa.cache_accept(cache, i32(table), ld, path.to(DEV), i32(list(counts)), n_q=i32(n_q), weights=wd if track else None,
                          lens_out=ld if alias else None)
    synced(fa)
    assert got.tolist() == want and (got is ld) == alias
    for name, t, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        np.testing.assert_array_equal(s.cpu().double().numpy(), ref.scale[name], err_msg=f"{name} scale")
        np.testing.assert_array_equal(R.stored(t.cpu()), ref.pool[name], err_msg=name)
    np.testing.assert_array_equal(wd.cpu().numpy(), want_w)


@pytest.mark.parametrize("kind", [E4M3, I8])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128), (256, 16), (128, 32)])
@pytest.mark.parametrize("n,counts", [(1, (1, 0, 1, 1)), (2, (1, 2, 0, 1)), (16, (4, 1, 16, 9)), (60, (3, 30, 59, 60)),
                                      (200, (1, 20, 100, 199))])
def test_accept(fa, kind, D, page, n, counts):
    """Drafts behind no token, at a block's end, in the middle; paths of one node to all."""
    accept_case(fa, kind=kind, D=D, page=page, n=n, counts=counts, lens=(n, n + page - 1, n + 77, n + 2 * page),
                alias=n == 16)


def test_accept_largest_and_padding(fa):
    accept_case(fa, n=1024, counts=(700, 1, 300), lens=(1024, 1400, 1100), kind=I8, D=128, page=64)
    accept_case(fa, n=12, n_q=(12, 5, 0, 1), counts=(3, 5, 0, 0), lens=(40, 30, 20, 10), track=False, alias=True)


def test_accept_paths_that_stay(fa):
    """Nothing moves where the path is the first drafts: no byte changes."""
    accept_case(fa, n=8, counts=(3, 8, 1), lens=(50, 64, 8), paths=[[0, 1, 2], list(range(8)), [0]])
    accept_case(fa, n=8, counts=(4, 2), lens=(50, 64), paths=[[0, 1, 6, 7], [0, 7]])


def test_accept_bad_entries(fa):
    """Paths that do not ascend or leave the drafts end there, counts are cut, sequences without their drafts stay, bad
    blocks are skipped; all told, and nothing else changes."""
    g = torch.Generator().manual_seed(2)
    lens, n = [40] * 6 + [3], 8
    table, P, _ = R.make_table(g, lens, 16)
    pools = R.make_pools(g, P, 1, 16, 64, E4M3)
    rows = [[0, 3, 3, 4], [0, 2, 8, 9], [-1, 2, 3, 4], [0, 1, 2, 3], [0, 2, 5, 6], [1, 0, 2, 3], [0, 1, 2, 3]]
    path = torch.full((7, n), -1, dtype=torch.int32)
    path[:, :4] = torch.tensor(rows)
    counts, good = [4, 4, 4, -2, 100, 4, 2], [2, 2, 0, 0, 4, 1, 0]
    n_q = [n] * 7
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    keep = [r[:k] for r, k in zip(rows, good)]
    want = T.accept(ref, table, lens, keep, good, n_q[:6] + [0])
    got = fa.cache_accept(cache, i32(table), i32(lens), path.to(DEV), i32(counts))
    told(fa)
    assert got.tolist() == want[:6] + [3]
    np.testing.assert_array_equal(R.stored(cache.k.cpu()), ref.pool["k"])
    np.testing.assert_array_equal(R.stored(cache.v.cpu()), ref.pool["v"])
    got = fa.cache_accept(cache, i32(table), i32(lens), path.to(DEV), i32([1] * 7), n_q=i32([9, -1, 8, 8, 8, 8, 3]))
    told(fa)
    assert got.tolist() == [40, 40, 32, 33, 33, 33, 1]
    bad = [list(r) for r in table]
    bad[0][2], bad[1][2] = P + 3, -1  # the block of both sequences' drafts
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v)]
    got = fa.cache_accept(cache, i32(bad)[:2], i32([40, 40]), i32([[0, 4], [0, 5]]), i32([2, 2]), n_q=i32([2, 2]))
    told(fa)  # (row 4 is outside two drafts)
    got = fa.cache_accept(cache, i32(bad)[:2], i32([40, 40]), path[4:6, :8].to(DEV), i32([4, 0]))
    told(fa)
    assert got.tolist() == [36, 32]
    for a, t in zip(before, (cache.k, cache.v)):
        assert torch.equal(a, t.view(torch.uint8))


def test_accept_of_drafts_that_the_table_has_no_room_for(fa):
    """Drafts behind the table were not appended: a path ends before the first of them, and the tokens before the drafts
    stay where they are; told."""
    g = torch.Generator().manual_seed(4)
    lens, n, page = [68, 100, 64, 66, 70], 8, 16
    table, P, _ = R.make_table(g, [64] * 5, page)
    pools = R.make_pools(g, P, 2, page, 64, E4M3)
    ref, cache = R.Cache(*pools), to_gpu(fa, pools)
    rows = [[0, 2, 5, 6], [0, 1, 2, 3], [0, 3, 4, 7], [0, 1, 3, 5], [2, 3, 4, 5]]
    path = torch.full((5, n), -1, dtype=torch.int32)
    path[:, :4] = torch.tensor(rows)
    n_q = [8, 8, 8, 7, 6]  # the drafts begin in slots 60, 92, 56, 59, 64
    w = torch.rand(5, 2, 70, generator=g)
    want_w, wd = w.numpy().copy(), w.to(DEV)
    kept = [[0, 2], [], rows[2], [0, 1, 3], []]
    want = T.accept(ref, table, [64] * 5, kept, [len(x) for x in kept], [4, 0, 8, 5, 0], want_w)
    got = fa.cache_accept(cache, i32(table), i32(lens), path.to(DEV), i32([4] * 5), n_q=i32(n_q), weights=wd)
    told(fa)
    assert got.tolist() == want == [62, 64, 60, 62, 64]
    np.testing.assert_array_equal(R.stored(cache.k.cpu()), ref.pool["k"])
    np.testing.assert_array_equal(R.stored(cache.v.cpu()), ref.pool["v"])
    np.testing.assert_array_equal(wd.cpu().numpy(), want_w)


# ----------------------------------------------------------------- together

def draft_loop(fa, steps=6, kind=E4M3, graph=False, stream=None):
    """Steps of one layer: append the drafts, attend, verify, accept.  Returns what each step gave, and the state."""
    g = torch.Generator().manual_seed(21)
    B, Hq, H, D, page, n, V, L0 = 3, 8, 2, 64, 16, 7, 500, 30
    M = -(-(L0 + (steps + 1) * n) // page)
    cache = fa.kv_cache(B * M, H, D, page=page, dtype=kind)
    table = torch.randperm(B * M, generator=g).to(torch.int32).view(B, M).to(DEV)
    W = M * page
    weights, positions = torch.zeros(B, H, W, device=DEV), torch.full((B, H, W), -1, dtype=torch.int32, device=DEV)
    lens = i32([0] * B)
    first = torch.randn(2, B, H, L0, D, generator=g).to(BF16).to(DEV)
    fa.cache_append(cache, first[0], first[1], table, lens, weights=weights, positions=positions)
    lens += L0
    rng = random.Random(5)
    draws = []
    for _ in range(steps):
        q, k, v = (torch.randn(B, h, n, D, generator=g).to(BF16) for h in (Hq, H, H))
        p = torch.softmax(torch.randn(B, n, V, generator=g) * 2, -1)
        z = torch.softmax(torch.log(p) + torch.randn(B, n, V, generator=g) * 0.5, -1)
        tree = torch.tensor([T.random_tree(rng, n, "beam") for _ in range(B)], dtype=torch.int32)
        tokens = torch.stack([torch.multinomial(z[b, tree[b].clamp_min(0).long()], 1, generator=g)[:, 0] for b in range(B)])
        draws.append([x.to(DEV) for x in (q, k, v, p, z, tree, tokens.to(torch.int32), torch.rand(B, n, generator=g),
                                          torch.rand(B, generator=g))])

    def step(q, k, v, p, z, tree, tokens, u, x):
        fa.cache_append(cache, k, v, table, lens, weights=weights, positions=positions)
        lens.add_(n)
        o, lse = fa.cache_attention(q, cache, table, lens, tree=tree, weights=weights)
        path, count, token = fa.verify_drafts(p, tokens, tree, u, x, p_draft=z)
        fa.cache_accept(cache, table, lens, path, count, weights=weights, lens_out=lens)
        return o, lse, path, count, token

    outs = []
    if not graph:
        for d in draws:
            outs.append(step(*d))
    else:
        hold = [x.clone() for x in draws[0]]
        state = [cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, weights, positions, lens]
        saved = [x.clone() for x in state]
        gr = torch.cuda.CUDAGraph()
        step(*hold)  # warm-up
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            o = step(*hold)
        for a, b in zip(state, saved):
            a.copy_(b)
        for d in draws:
            for a, b in zip(hold, d):
                a.copy_(b)
            gr.replay()
            outs.append(tuple(x.clone() for x in o))
    synced(fa)
    return outs, draws, (cache, table, weights, positions, lens, first)


@pytest.mark.parametrize("kind", [E4M3, I8])
def test_draft_loop_against_plain_decoding(fa, kind):
    """The cache holds what the accepted tokens would have left behind if only they had been appended: the same stored
    values times their scales in e4m3 (powers of two keep its bits), a step apart in int8; positions in order."""
    outs, draws, (cache, table, weights, positions, lens, first) = draft_loop(fa, kind=kind)
    B, page = 3, 16
    assert max(o[3].max().item() for o in outs) > 2
    for b in range(B):
        ks = [first[0][b]]
        for (q, k, *_), (o, lse, path, count, token) in zip(draws, outs):
            ks.append(k[b][:, path[b, :count[b]].long()])
        k = torch.cat(ks, 1)  # [H, L, D]
        L = lens[b].item()
        assert k.shape[1] == L
        pages = table[b, :-(-L // page)].long()
        got = (cache.k[pages].float() * cache.k_scale[pages][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
        step = cache.k_scale[pages].repeat_interleave(page, 0)[:L].T[..., None]
        if kind == E4M3:  # half a step: 2^-4 of the value, or half the least denormal
            tol = torch.maximum(k.float().abs() * 2.0 ** -4, step * 2.0 ** -10)
        else:  # a rounding at each of the sizes that its block's scale had: half a step of each, 1/2 + 1/4 + ..
            tol = step
        assert ((got - k.float()).abs() <= tol).all()
        assert positions[b, 0, :L].tolist() == list(range(L))
    assert torch.isfinite(weights).all()


def test_draft_loop_in_a_graph(fa):
    """A captured step follows lengths, paths and trees that change between replays."""
    a, _, sa = draft_loop(fa)
    b, _, sb = draft_loop(fa, graph=True)
    for x, y in zip(a, b):
        for s, t in zip(x, y):
            assert torch.equal(s, t)
    for s, t in zip((sa[0].k_scale, sa[2], sa[3], sa[4]), (sb[0].k_scale, sb[2], sb[3], sb[4])):
        assert torch.equal(s, t)


def test_draft_loop_on_another_stream(fa):
    a, _, sa = draft_loop(fa)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, _, sb = draft_loop(fa)
    s.synchronize()
    for x, y in zip(a, b):
        for p, q in zip(x, y):
            assert torch.equal(p, q)


def test_draft_operators_on_a_raw_stream(fa):
    """`stream`: what is allocated belongs to it; results as on the current one."""
    s = torch.cuda.Stream()
    p = torch.softmax(torch.randn(2, 3, 50, device=DEV), -1)
    tokens, tree, u, x = i32([[0, 1, 2]] * 2), i32([-1, 0, 0]), torch.rand(2, 3, device=DEV), torch.rand(2, device=DEV)
    torch.cuda.synchronize()
    want = fa.verify_drafts(p, tokens, tree, u, x)
    got = fa.verify_drafts(p, tokens, tree, u, x, stream=s.cuda_stream)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    cache = fa.kv_cache(2, 1, 64, page=16)
    lens = fa.cache_accept(cache, i32([[0], [1]]), i32([5, 9]), got[0], got[1], stream=s.cuda_stream)
    s.synchronize()
    assert lens.tolist() == [2 + got[1][0].item(), 6 + got[1][1].item()]


def test_two_calls_at_once(fa):
    """The same operators on two streams, each with its own scratch and outputs."""
    want = draft_loop(fa)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            got.append(draft_loop(fa)[0])
    torch.cuda.synchronize()
    for outs in got:
        for x, y in zip(want, outs):
            for p, q in zip(x, y):
                assert torch.equal(p, q)


def test_python_refusals(fa):
    cache = fa.kv_cache(4, 2, 64, page=16)
    table, lens, q = i32([[0, 1]]), i32([20]), torch.zeros(1, 4, 3, 64, dtype=BF16, device=DEV)
    tree = i32([-1, 0, 0])
    fa.cache_attention(q, cache, table, lens, tree=tree)
    for kw, needle in ((dict(tree=tree.long()), "tree"), (dict(tree=tree[:2]), "tree"), (dict(tree=tree.cpu()), "tree"),
                       (dict(tree=i32([[-1, 0, 0]] * 2)), "tree"), (dict(tree=tree, causal=False), "causal"),
                       (dict(tree=torch.stack([tree, tree], 1)[:, 0]), "unit stride")):
        with pytest.raises(ValueError, match=needle):
            fa.cache_attention(q, cache, table, lens, **kw)
    with pytest.raises(fa.FaError, match="1024"):
        fa.cache_attention(torch.zeros(1, 2, 1025, 64, dtype=BF16, device=DEV), cache, table, lens, tree=i32([-1] * 1025))
    p, u, x = torch.ones(1, 3, 8, device=DEV), torch.zeros(1, 3, device=DEV), torch.zeros(1, device=DEV)
    t = i32([[0, 1, 2]])
    for a, needle in (((p.double(), t, tree, u, x), "dtype"), ((p[0], t, tree, u, x), "3-D"), ((p, t.long(), tree, u, x), "tokens"),
                      ((p, t, tree, u.double(), x), "u must"), ((p, t, tree, u, u), "u_next"), ((p, t[:, :2], tree, u, x), "tokens"),
                      ((p.transpose(1, 2), t, tree, u, x), "unit stride"), ((p[:, :0], t[:, :0], tree[:0], u[:, :0], x), "> 0")):
        with pytest.raises(ValueError, match=needle):
            fa.verify_drafts(*a)
    with pytest.raises(ValueError, match="p_draft"):
        fa.verify_drafts(p, t, tree, u, x, p_draft=p.to(BF16))
    path, count = i32([[0, 1, -1]]), i32([2])
    for a, kw, needle in (((path.long(), count), {}, "path"), ((path[0], count), {}, "path"), ((path, count.long()), {}, "count"),
                          ((path, count), dict(n_q=count.cpu()), "n_q"), ((path, count), dict(weights=u), "weights"),
                          ((path, count), dict(lens_out=x), "lens_out"), ((path[:, :0], count), {}, "at least one")):
        with pytest.raises(ValueError, match=needle):
            fa.cache_accept(cache, table, lens, *a, **kw)
    assert fa.verify_drafts(p[:0], t[:0], tree, u[:0], x[:0])[0].shape == (0, 3)
    synced(fa)
