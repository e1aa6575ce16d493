"""Host-side tests of the serving operators' C ABI and Python layer (no GPU needed): include/fa_cache.h and the
library agree, argument structs match the header, and bad arguments are refused before any CUDA call."""
import copy
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import cache_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fa_cache.h")
P = 0x10000  # a stand-in address: validation never follows it


@pytest.fixture(scope="module")
def fa():
    from attention_forward_08_gb300 import _build
    _build.build()
    import attention_forward_08_gb300 as fa
    fa.load_library()
    return fa


def test_header_and_exports(fa):
    names = sorted(set(re.findall(r"^\s*(?:int|long long)\s+(fa_\w+)\s*\(", open(HEADER).read(), re.M)))
    assert names == sorted(fa.cache.CACHE_EXPORTED)
    for name in names:
        assert hasattr(fa.load_library(), name)


@pytest.mark.parametrize("cname,pyname", [("fa_cache", "FaCache"), ("fa_cache_append_args", "FaCacheAppendArgs"),
                                          ("fa_cache_attn_args", "FaCacheAttnArgs"),
                                          ("fa_cache_evict_args", "FaCacheEvictArgs")])
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


def cache_struct(fa, **kw):
    c = fa.FaCache()
    c.k = c.v = c.k_scale = c.v_scale = P
    c.P, c.H_kv, c.page, c.D, c.kind = 8, 2, 64, 128, 0
    c.k_strides[:] = c.v_strides[:] = (2 * 64 * 128, 64 * 128, 128)
    for k, v in kw.items():
        if k.endswith("strides"):
            getattr(c, k)[:] = v
        else:
            setattr(c, k, v)
    return c


def args_of(fa, which, cache=None, **kw):
    S = {"append": fa.FaCacheAppendArgs, "attn": fa.FaCacheAttnArgs, "evict": fa.FaCacheEvictArgs}[which]
    a = S()
    a.cache = cache_struct(fa, **(cache or {}))
    a.table, a.table_stride, a.lens, a.B, a.M = P, 4, P, 2, 4
    if which == "append":
        a.k = a.v = P
        a.n, a.dtype = 3, 1
        a.k_strides[:] = a.v_strides[:] = (2 * 3 * 128, 3 * 128, 128)
    elif which == "attn":
        a.q = a.o = a.lse = P
        a.H_q, a.n, a.scale, a.dtype = 8, 1, 0.1, 1
        a.q_strides[:] = a.o_strides[:] = (8 * 128, 128, 128)
        a.workspace, a.workspace_bytes = P, 1 << 40
    else:
        a.weights = a.positions = a.lens_out = P
        a.W, a.keep, a.recent = 256, 64, 8
        a.workspace, a.workspace_bytes = P, 1 << 40
    for k, v in kw.items():
        if k.endswith("strides"):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


COMMON = [
    (dict(cache=dict(k=None)), 1, "non-NULL"),
    (dict(cache=dict(v_scale=None)), 1, "non-NULL"),
    (dict(cache=dict(P=0)), 1, "> 0"),
    (dict(cache=dict(H_kv=-1)), 1, "> 0"),
    (dict(cache=dict(kind=2)), 1, "kind"),
    (dict(cache=dict(page=48)), 2, "page"),
    (dict(cache=dict(page=256)), 2, "page"),
    (dict(cache=dict(D=96)), 2, "head dim"),
    (dict(cache=dict(v=P + 8)), 3, "16-byte"),
    (dict(cache=dict(k_scale=P + 2)), 3, "4-byte"),
    (dict(cache=dict(k_strides=(16384, 8192, 120))), 3, "strides"),
    (dict(cache=dict(v_strides=(16384, -8192, 128))), 3, "strides"),
    (dict(table=None), 1, "table"),
    (dict(lens=None), 1, "lens"),
    (dict(B=0), 1, "> 0"),
    (dict(M=0), 1, "> 0"),
    (dict(M=1 << 30, table_stride=1 << 30), 2, "2^31"),
    (dict(B=70000), 2, "65535"),
    (dict(table_stride=3), 1, "row stride"),
    (dict(lens=P + 1), 3, "4-byte"),
]


@pytest.mark.parametrize("which", ["append", "attn", "evict"])
@pytest.mark.parametrize("kw,status,needle", COMMON)
def test_common_refusals(fa, which, kw, status, needle):
    a = args_of(fa, which, **kw)
    assert getattr(fa, "fa_cache_" + which)(a) == status
    assert needle in fa.fa_last_error()


@pytest.mark.parametrize("which,kw,status,needle", [
    ("append", dict(k=None), 1, "non-NULL"),
    ("append", dict(n=0), 1, "n (0)"),
    ("append", dict(dtype=5), 1, "dtype"),
    ("append", dict(v=P + 4), 3, "16-byte"),
    ("append", dict(weights=P, W=0), 1, "W must"),
    ("append", dict(seen=P + 2), 3, "4-byte"),
    ("append", dict(k_strides=(768, 384, 64)), 3, "strides"),
    ("append", dict(v_strides=(768, 385, 128)), 3, "strides"),
    ("attn", dict(q=None), 1, "non-NULL"),
    ("attn", dict(lse=None), 1, "non-NULL"),
    ("attn", dict(n=0), 1, "n (0)"),
    ("attn", dict(H_q=7), 1, "divisible"),
    ("attn", dict(dtype=0), 2, "dtype"),
    ("attn", dict(dtype=9), 1, "dtype"),
    ("attn", dict(scale=float("nan")), 1, "finite"),
    ("attn", dict(window=-1), 1, "window"),
    ("attn", dict(softcap=-1.0), 1, "softcap"),
    ("attn", dict(softcap=float("inf")), 1, "softcap"),
    ("attn", dict(weights=P, W=0), 1, "W must"),
    ("attn", dict(weights=P + 1, W=4), 3, "4-byte"),
    ("attn", dict(n=1 << 28), 2, "2^31"),
    ("attn", dict(q=P + 2), 3, "16-byte"),
    ("attn", dict(o_strides=(1024, 130, 128)), 3, "strides"),
    ("evict", dict(weights=None), 1, "non-NULL"),
    ("evict", dict(lens_out=None), 1, "non-NULL"),
    ("evict", dict(W=0), 1, "W must"),
    ("evict", dict(keep=0), 1, "keep"),
    ("evict", dict(recent=65), 1, "recent"),
    ("evict", dict(recent=-1), 1, "recent"),
    ("evict", dict(positions=None), 1, "positions"),
    ("evict", dict(into=P, M_into=0), 1, "into"),
    ("evict", dict(into=P, M_into=1, keep=65), 1, "into"),
    ("evict", dict(into=P, M_into=2, into_stride=1), 1, "into"),
    ("evict", dict(into=P, M_into=1, into_stride=1, weights_out=P, W_out=63), 1, "W_out"),
    ("evict", dict(keep=1 << 30), 2, "2^31"),
    ("evict", dict(workspace=None), 1, "workspace"),
    ("evict", dict(workspace=P + 16), 3, "256-byte"),
    ("evict", dict(workspace_bytes=100), 1, "smaller"),
])
def test_refusals(fa, which, kw, status, needle):
    a = args_of(fa, which, **kw)
    assert getattr(fa, "fa_cache_" + which)(a) == status
    assert needle in fa.fa_last_error()
    if which != "append" and "workspace" not in "".join(kw):
        assert getattr(fa, f"fa_cache_{which}_workspace_bytes")(a) == -1


def test_null_args(fa):
    lib = fa.cache._library()
    for name in ("fa_cache_append", "fa_cache_attn", "fa_cache_evict"):
        assert getattr(lib, name)(None) == 1 and "NULL" in fa.fa_last_error()


def test_evict_workspace_size(fa):
    """Slots named per head twice (4 bytes each), and a count per head."""
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    a = args_of(fa, "evict", B=3, keep=100, table_stride=4)
    assert fa.fa_cache_evict_workspace_bytes(a) == 2 * up(3 * 2 * 100 * 4) + up(3 * 2 * 4)


def test_python_refuses_cpu_tensors_and_bad_pools(fa):
    k = torch.zeros(4, 2, 64, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.KVCache(k, k, s, s)
    with pytest.raises(ValueError, match="dtype"):
        fa.KVCache(k.view(torch.uint8), k, s, s)
    with pytest.raises(ValueError, match="v must"):
        fa.KVCache(k, k[:2], s, s)
    with pytest.raises(ValueError, match="k_scale"):
        fa.KVCache(k, k, s[:, :1], s)
    with pytest.raises(ValueError, match="unit stride"):
        fa.KVCache(k.transpose(2, 3), k.transpose(2, 3), s, s)

def test_python_cache_keeps_its_tensors(fa):
    """Calls use the addresses that the cache was made with: other tensors are refused, not ignored."""
    cache = fa.KVCache.__new__(fa.KVCache)
    for name in ("k", "v", "k_scale", "v_scale", "c", "device"):
        with pytest.raises(AttributeError, match="KVCache"):
            setattr(cache, name, torch.zeros(1))
    assert copy.copy(cache) is cache


# ----------------------------------------------------------------- the reference itself

def test_reference_rounding_is_torchs():
    x = torch.cat([torch.randn(4000, dtype=torch.float64) * 10.0 ** e for e in range(-4, 3)])
    x = torch.cat([x, torch.arange(-64, 64, dtype=torch.float64) / 1024])  # the denormals and halves between them
    np.testing.assert_array_equal(R.round8(x.numpy(), R.E4M3), x.clamp(-448, 448).float().to(R.E4M3).double().numpy())


def test_reference_attention_is_a_softmax():
    g = torch.Generator().manual_seed(0)
    pools = R.make_pools(g, 3, 1, 16, 64, R.E4M3)
    c = R.Cache(*pools)
    q = torch.randn(1, 2, 3, 64, generator=g)
    o, lse, w, _, _ = R.attention(c, q, [[2, 0, 1]], [40], causal=True)
    k, v = (torch.cat([(x[i].double() * s[i].double()[:, None, None])[0] for i in (2, 0, 1)])[:40]
            for x, s in ((pools[0], pools[2]), (pools[1], pools[3])))
    s = q[0].double() @ k.T / 8
    s[:, torch.arange(40)[None] > 37 + torch.arange(3)[:, None]] = -float("inf")
    np.testing.assert_allclose(o[0], (s.softmax(-1) @ v).numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse[0], s.logsumexp(-1).numpy(), rtol=1e-12)
    np.testing.assert_allclose(w[0, 0], s.softmax(-1).sum((0, 1)).numpy(), rtol=1e-12, atol=1e-15)
