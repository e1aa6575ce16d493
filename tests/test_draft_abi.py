"""Host-side tests of decoding with drafts (no GPU needed): argument structs match include/fa_cache.h, bad arguments
are refused before any CUDA call, and the definition that the GPU tests compare with does what it is for."""
import ctypes
import itertools
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import cache_reference as R
import draft_reference as D
from test_cache_abi import COMMON, P, args_of, cache_struct

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fa():
    from attention_forward_08_gb300 import _build
    _build.build()
    import attention_forward_08_gb300 as fa
    fa.load_library()
    return fa


@pytest.mark.parametrize("cname,pyname", [("fa_cache_attn_tree_args", "FaCacheAttnTreeArgs"),
                                          ("fa_verify_drafts_args", "FaVerifyDraftsArgs"),
                                          ("fa_cache_accept_args", "FaCacheAcceptArgs")])
def test_structs_match_header(fa, tmp_path, cname, pyname):
    S = getattr(fa, pyname)
    fields = [f for f, _ in S._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "fa_cache.h"\nint main(void){\n'
                   f'  printf("%zu\\n", sizeof({cname}));\n'
                   + "".join(f'  printf("%zu\\n", offsetof({cname}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(tmp_path / "layout")], check=True)
    vals = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    assert vals == [ctypes.sizeof(S)] + [getattr(S, f).offset for f in fields]


def draft_args(fa, which, **kw):
    if which == "tree":
        own = {k: kw.pop(k) for k in ("tree", "tree_stride") if k in kw}
        a = fa.FaCacheAttnTreeArgs()
        a.attn = args_of(fa, "attn", **{"causal": 1, **kw})
        a.tree, a.tree_stride = own.get("tree", P), own.get("tree_stride", a.attn.n)
        return a
    if which == "verify":
        a = fa.FaVerifyDraftsArgs()
        a.p = a.q = a.tokens = a.tree = a.u = a.u_next = a.path = a.count = a.token = P
        a.p_strides[:] = a.q_strides[:] = (400, 100)
        a.tokens_stride = a.tree_stride = a.u_stride = 4
        a.B, a.n, a.V, a.dtype = 2, 4, 100, 0
    else:
        a = fa.FaCacheAcceptArgs()
        a.cache = cache_struct(fa, **kw.pop("cache", {}))
        a.table, a.table_stride, a.lens, a.B, a.M = P, 4, P, 2, 4
        a.path, a.path_stride, a.count, a.lens_out, a.n = P, 5, P, P, 5
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def call(fa, which):
    return {"tree": fa.fa_cache_attn_tree, "verify": fa.fa_verify_drafts, "accept": fa.fa_cache_accept}[which]


@pytest.mark.parametrize("which", ["tree", "accept"])
@pytest.mark.parametrize("kw,status,needle", COMMON)
def test_common_refusals(fa, which, kw, status, needle):
    assert call(fa, which)(draft_args(fa, which, **dict(kw))) == status
    assert needle in fa.fa_last_error()


@pytest.mark.parametrize("which,kw,status,needle", [
    ("tree", dict(q=None), 1, "non-NULL"),
    ("tree", dict(n=0), 1, "n (0)"),
    ("tree", dict(tree=None), 1, "tree"),
    ("tree", dict(tree=P + 2), 3, "4-byte"),
    ("tree", dict(n=8, tree_stride=7), 1, "row stride"),
    ("tree", dict(n=8, tree_stride=-8), 1, "row stride"),
    ("tree", dict(n=1025), 2, "1024"),
    ("tree", dict(causal=0), 1, "causal"),
    ("tree", dict(dtype=0), 2, "dtype"),
    ("tree", dict(window=-2), 1, "window"),
    ("verify", dict(p=None), 1, "non-NULL"),
    ("verify", dict(tokens=None), 1, "non-NULL"),
    ("verify", dict(u_next=None), 1, "non-NULL"),
    ("verify", dict(token=None), 1, "non-NULL"),
    ("verify", dict(tree=None), 1, "tree"),
    ("verify", dict(B=0), 1, "> 0"),
    ("verify", dict(n=-1), 1, "> 0"),
    ("verify", dict(V=0), 1, "> 0"),
    ("verify", dict(dtype=3), 1, "dtype"),
    ("verify", dict(B=65536), 2, "65535"),
    ("verify", dict(V=(1 << 20) + 1), 2, "1048576"),
    ("verify", dict(n=1025, tree_stride=1025), 2, "1024"),
    ("verify", dict(tree_stride=3), 1, "row stride"),
    ("verify", dict(p=P + 2), 3, "elements"),
    ("verify", dict(q=P + 1, dtype=1), 3, "elements"),
    ("verify", dict(count=P + 1), 3, "4-byte"),
    ("accept", dict(path=None), 1, "non-NULL"),
    ("accept", dict(lens_out=None), 1, "non-NULL"),
    ("accept", dict(n=0), 1, "n (0)"),
    ("accept", dict(n=1025, path_stride=1025), 2, "1024"),
    ("accept", dict(path_stride=4), 1, "row stride"),
    ("accept", dict(weights=P, W=0), 1, "W must"),
    ("accept", dict(weights=P + 2, W=10), 3, "4-byte"),
])
def test_refusals(fa, which, kw, status, needle):
    a = draft_args(fa, which, **dict(kw))
    assert call(fa, which)(a) == status
    assert needle in fa.fa_last_error()
    if which == "tree":
        assert fa.fa_cache_attn_tree_workspace_bytes(a) == -1


APART = dict(lens=P + 64, count=P + 4096, path=P + 8192, table=P + 12288)  # (2 sequences, 5 drafts, 4 blocks)


@pytest.mark.parametrize("kw", [dict(lens_out=P + 64 + 4), dict(lens_out=P + 64 - 4), dict(lens_out=P + 4096),
                                dict(lens_out=P + 4096 - 4), dict(n_q=P + 16384, lens_out=P + 16384 + 4),
                                dict(lens_out=P + 8192 + 36), dict(path_stride=9, lens_out=P + 8192 + 52),
                                dict(lens_out=P + 12288 + 28), dict(lens_out=P + 64, n_q=P + 68)])
def test_accept_refuses_lengths_over_what_it_reads(fa, kw):
    """Blocks of a sequence read its numbers while one of them writes lens_out."""
    assert fa.fa_cache_accept(draft_args(fa, "accept", **{**APART, **kw})) == 1
    assert "share no memory" in fa.fa_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are stand-ins")
@pytest.mark.parametrize("lens_out", [P + 64, P + 64 + 8, P + 64 - 8, P + 4096 - 8, P + 8192 + 40, P + 12288 + 32])
def test_accept_takes_lengths_that_are_lens_or_apart(fa, lens_out):
    for n_q in (None, P + 64):
        fa.fa_cache_accept(draft_args(fa, "accept", **APART, lens_out=lens_out, n_q=n_q if lens_out == P + 64 else None))
        assert "share no memory" not in fa.fa_last_error()  # (there is no device)


def test_null_args(fa):
    lib = fa.cache._library()
    for name in ("fa_cache_attn_tree", "fa_verify_drafts", "fa_cache_accept"):
        assert getattr(lib, name)(None) == 1 and "NULL" in fa.fa_last_error()


def test_python_refuses_cpu_tensors(fa):
    p, i, u = torch.ones(1, 2, 4), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.verify_drafts(p, i, i, u, u[:, 0])
    with pytest.raises(ValueError, match="3-D"):
        fa.verify_drafts(p[0], i, i, u, u[:, 0])


# ----------------------------------------------------------------- the reference itself

@pytest.mark.parametrize("window", [0, 1, 5, 40])
def test_reference_chain_is_causal(window):
    g = torch.Generator().manual_seed(0)
    pools = R.make_pools(g, 4, 2, 16, 64, R.E4M3)
    c = R.Cache(*pools)
    q = torch.randn(2, 4, 6, 64, generator=g)
    table, lens = [[2, 0, 3], [1, -1, -1]], [40, 4]
    chain = [D.random_tree(random.Random(0), 6, "chain")] * 2
    for got, want in zip(D.attention(c, q, table, lens, chain, window=window),
                         R.attention(c, q, table, lens, window=window)):
        np.testing.assert_allclose(got, want, rtol=1e-13)


def test_reference_siblings_do_not_see_each_other():
    see = D.visible([-1, 0, 0, 2, 1], 9, 5)
    assert see[:, :4].all()
    assert see[:, 4:].tolist() == [[True, False, False, False, False], [True, True, False, False, False],
                                   [True, False, True, False, False], [True, False, True, True, False],
                                   [True, True, False, False, True]]
    see = D.visible([-1, 0, 0, 2, 1], 9, 5, window=2)  # positions 4, 5, 5, 6, 6
    assert np.argwhere(see).tolist() == [[0, 3], [0, 4], [1, 4], [1, 5], [2, 4], [2, 6], [3, 6], [3, 7], [4, 5], [4, 8]]


@pytest.mark.parametrize("drawn", [True, False])
def test_rule_keeps_the_target_distribution(drawn):
    """Two children of one node, every draw and every outcome by its probability: the token behind the node has the
    target's distribution, to 64 bits."""
    rng = np.random.default_rng(1)
    V = 4
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    got = np.zeros(V)
    draws = itertools.product(range(V), repeat=2) if drawn else [(2, 0)]
    for ts in draws:
        left = D.residuals(p, q if drawn else None, ts)
        chance = q[ts[0]] * q[ts[1]] if drawn else 1.0
        for t, (r, z) in zip(ts, left):
            yes = min(1.0, r[t] / ((q[t] if drawn else 1.0) * z))  # P(u q Z < r)
            got[t] += chance * yes
            chance *= 1.0 - yes
        r, _ = left[-1]
        got += chance * r / r.sum()
    np.testing.assert_allclose(got, p, rtol=1e-12)


def test_reference_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.2, 0.3, 0.5]])
    q = np.array([[0.25, 0.5, 0.25], [1.0, 0.0, 0.0], [1.0, 0.0, 0.0]])
    # node 1 (token 1): 0.6 * 0.5 < 0.25 does not hold; r = (0.25, 0, 0), Z = 0.25; node 2 (token 0): 0.5 * 0.25 * 0.25 < 0.25
    assert D.verify(p, [0, 1, 0], [-1, 0, 0], [0.0, 0.6, 0.5], 0.35, q) == ([0, 2], 1)
    assert D.verify(p, [0, 1, 2], [-1, 0, 0], [0.0, 0.6, 0.5], 0.99, q) == ([0], 0)
    # candidates: 0.3 < 0.25 does not hold, Z = 0.75, 0.3 * 0.75 < 0.25 holds
    assert D.verify(p, [0, 1, 2], [-1, 0, 0], [0.0, 0.3, 0.3], 0.6) == ([0, 2], 2)
    assert D.verify(p, [0, 1, 1], [-1, 0, 0], [0.0, 0.3, 0.0], 0.7) == ([0], 2)  # r = (0.5, 0, 0.25)
