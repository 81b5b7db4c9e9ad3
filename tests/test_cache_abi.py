"""The 8-bit cache's boundary without a GPU: exports, refusals on the host, the reference's own pins."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import cache_reference as ref
from io_aware_exact_fa2_gb300 import build as fa2_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CUDA_ERR = 0, 1, 2, 3
P = 0x10000   # fake, never dereferenced, aligned


@pytest.fixture(scope="module")
def lib():
    fa2_build.build()
    from io_aware_exact_fa2_gb300 import _cache_binding
    return _cache_binding


def header_functions():
    text = open(os.path.join(ROOT, "include", "fa2_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fa2_\w+)\s*\(", text)))


def test_library_exports_what_its_header_declares(lib):
    for name in header_functions():
        assert hasattr(lib._lib, name), name
    if shutil.which("nm"):
        out = subprocess.run(["nm", "-D", "--defined-only", lib.cache_library_path()], capture_output=True, text=True,
                             check=True).stdout
        exported = sorted({x.split()[-1] for x in out.splitlines() if x.split() and x.split()[-2] in "TWDB"})
        assert exported == header_functions()


class Cache(ctypes.Structure):
    """struct fa2_cache, the stride arrays as single fields."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table")] +
                [(n, ctypes.c_longlong) for n in ("k_page", "k_head", "k_slot", "v_page", "v_head", "v_slot")] +
                [(n, ctypes.c_int) for n in ("num_pages", "H", "page_size", "D", "B", "max_pages")])


def cache(lib, **kw):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, page_table=P, num_pages=4, H=2, page_size=16, D=64, B=1, max_pages=2)
    f.update(kw)
    return bytes(Cache(**f))


def ll3(*x):
    return bytes((ctypes.c_longlong * 3)(*x))


def test_the_binding_packs_the_structure(lib):
    c = Cache(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17)
    assert bytes(c) == lib._pack_cache(*range(1, 18))


def write(lib, c, k=P, v=P, ks=None, vs=None, starts=P, counts=None, L=5, f="fa2_cache_write"):
    return getattr(lib._lib, f)(c, k, v, ks, vs, starts, counts, L, None)


def attn(lib, c, q=P, o=P, lse=P, qs=None, os_=None, kv=P, ql=None, Hq=4, Lq=1, causal=1, window=-1, scale=0.1, ws=None,
         n=0):
    return lib._lib.fa2_cache_attn(c, q, o, lse, qs, os_, kv, ql, Hq, Lq, causal, window, scale, ws, n, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k_scale=0), INVALID), (dict(v_scale=0), INVALID),
    (dict(page_table=0), INVALID), (dict(k=P + 8), INVALID), (dict(v=P + 1), INVALID), (dict(page_table=P + 2), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=-1), INVALID), (dict(D=0), INVALID), (dict(page_size=0), INVALID),
    (dict(B=65536, H=65536), INVALID), (dict(max_pages=1 << 28), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(D=512), UNSUPPORTED),
    (dict(k_page=2048, k_head=1024, k_slot=72), INVALID), (dict(v_page=2048, v_head=0, v_slot=64), INVALID),
    (dict(k_page=-2048, k_head=1024, k_slot=64), INVALID), (dict(k_page=(1 << 38) + 16, k_head=1024, k_slot=64), INVALID),
])
def test_a_bad_cache_is_refused_by_every_entry_point(lib, kw, expect):
    c = cache(lib, **kw)
    assert write(lib, c) == expect
    assert write(lib, c, f="fa2_cache_read") == expect
    if kw.get("H") != 0:
        assert attn(lib, c, Hq=max(4, kw.get("H", 2))) == expect
    assert lib._lib.fa2_cache_write(None, P, P, None, None, P, None, 1, None) == INVALID


@pytest.mark.parametrize("kw,expect", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k=P + 2), INVALID), (dict(v=P + 8), INVALID),
    (dict(starts=0), INVALID), (dict(starts=P + 1), INVALID), (dict(counts=P + 2), INVALID),
    (dict(L=-1), INVALID), (dict(L=(1 << 30) + 1), INVALID), (dict(ks=ll3(640, 320, 60)), INVALID),
    (dict(vs=ll3(640, 0, 64)), INVALID), (dict(vs=ll3(-640, 320, 64)), INVALID), (dict(L=0), OK),
])
def test_bad_moves_are_refused(lib, kw, expect):
    for f in ("fa2_cache_write", "fa2_cache_read"):
        assert write(lib, cache(lib), f=f, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(lse=0), INVALID), (dict(kv=0), INVALID),
    (dict(q=P + 8), INVALID), (dict(o=P + 2), INVALID), (dict(lse=P + 2), INVALID), (dict(kv=P + 1), INVALID),
    (dict(ql=P + 2), INVALID), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hq=-2), INVALID), (dict(Lq=-1), INVALID),
    (dict(Lq=1 << 30), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(window=-2), INVALID),
    (dict(window=3, causal=0), INVALID), (dict(qs=ll3(256, 64, 4)), INVALID), (dict(os_=ll3(0, 64, 64)), INVALID),
    (dict(ws=P + 16, n=1 << 30), INVALID), (dict(Lq=0), OK),
])
def test_bad_attention_arguments_are_refused(lib, kw, expect):
    assert attn(lib, cache(lib), **kw) == expect


def test_workspace_size_refusals(lib):
    n = ctypes.c_size_t(7)
    f = lib._lib.fa2_cache_attn_workspace_size
    assert f(1, 4, 2, 1, 64, 0, None) == INVALID
    for bad in ((0, 4, 2, 1, 64, 0), (1, 4, 3, 1, 64, 0), (1, 0, 2, 1, 64, 0), (1, 4, 2, -1, 64, 0), (1, 4, 2, 1, 64, -1)):
        assert f(*bad, ctypes.byref(n)) == INVALID and n.value == 0
    assert f(1, 4, 2, 1, 80, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(1, 4, 2, 0, 64, 0, ctypes.byref(n)) == OK and n.value == 0


def test_without_a_gpu_the_calls_say_so(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; this checks the no-device path")
    assert write(lib, cache(lib)) == CUDA_ERR
    assert attn(lib, cache(lib)) == CUDA_ERR


def tensors(B=1, H=2, Pg=16, D=64, N=4, M=2, Lq=1, Hq=4):
    z = torch.zeros
    return dict(q=z(B, Hq, Lq, D, dtype=torch.bfloat16), k_cache=z(N, H, Pg, D).to(torch.float8_e4m3fn),
                v_cache=z(N, H, Pg, D).to(torch.float8_e4m3fn), k_scale=z(N, H, dtype=torch.uint8),
                v_scale=z(N, H, dtype=torch.uint8), page_table=z(B, M, dtype=torch.int32),
                kv_lens=z(B, dtype=torch.int32), o=z(B, Hq, Lq, D, dtype=torch.bfloat16), lse=z(B, Hq, Lq))


def test_binding_refuses_what_it_can_see(lib):
    from io_aware_exact_fa2_gb300 import fa2_cache_attn, fa2_cache_write
    t = tensors()
    with pytest.raises(ValueError):     # not on a GPU
        fa2_cache_attn(**t)
    for name, bad, error in (("k_cache", t["k_cache"].view(torch.uint8), TypeError),
                             ("v_cache", t["v_cache"][:, :1], ValueError),
                             ("k_cache", t["k_cache"][0], ValueError)):
        with pytest.raises(error):
            fa2_cache_attn(**{**t, name: bad})
    with pytest.raises((ValueError, TypeError)):
        fa2_cache_write(t["q"], t["q"], t["k_cache"].float(), t["v_cache"], t["k_scale"], t["v_scale"], t["page_table"],
                        t["kv_lens"])


# ------------------------------------------------- the reference's own pins

def test_reference_codes_are_torchs():
    every = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.decode(every), t)
    x = np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.random.default_rng(1).integers(-12, 9, 4000)
    x = np.concatenate([x, ref._CODES[:127], (ref._CODES[:126] + ref._CODES[1:127]) / 2]).clip(-448, 448)
    want = torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.encode(x.astype(np.float32)), want)
    np.testing.assert_array_equal(ref.encode([np.inf, -np.inf, np.nan, 1e9, -1e9]), [0x7f, 0x7f, 0x7f, 0x7e, 0xfe])


def test_reference_write_keeps_every_value_near():
    """Tokens appended one by one, growing: every code stays within a rounding, and one more
    where a grown scale made it subnormal, of its value."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 1, 40, 64)) * 2.0 ** (np.arange(40) / 4)[None, None, :, None]
    x = ref.bf16(x).double().numpy()
    codes, scale = np.zeros((3, 1, 16, 64), np.uint8), np.zeros((3, 1), np.uint8)
    table = np.array([[2, 0, 1]])
    for i in range(40):
        ref.write(x[:, :, i:i + 1], codes, scale, table, [i], [1])
        got, there = ref.gather(codes, scale, table[0], 0, i + 1)
        assert there.all()
        p = scale[table[0, : i // 16 + 1], 0].astype(float) - 127
        step = np.repeat(2.0 ** p, 16)[: i + 1, None] * 2.0 ** -9
        assert np.all(np.abs(got - x[0, 0, : i + 1]) <= 2.0 ** -4 * np.abs(x[0, 0, : i + 1]) + step)


def test_reference_scale_is_the_least_that_holds_the_largest():
    for top, e in ((448.0, 0), (449.0, 1), (450.0, 1), (447.0, 0), (1.75, -8), (1.76, -7), (2.0, -7), (0.0, -96),
                   (2.0 ** -100, -96), (3.3e38, 119), (np.inf, -96)):
        x = np.zeros((1, 1, 1, 64))
        x[..., 5] = top
        codes, scale = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.uint8)
        ref.write(x, codes, scale, np.zeros((1, 1), int), [0], [1])
        assert int(scale[0, 0]) - 127 == e, top


def test_reference_attention_against_torch():
    g = torch.Generator().manual_seed(0)
    B, H, G, Lq, n, D, Pg = 2, 2, 3, 5, 37, 64, 16
    k = torch.randn(B, H, 48, D, generator=g).to(torch.float8_e4m3fn)
    v = torch.randn(B, H, 48, D, generator=g).to(torch.float8_e4m3fn)
    q = torch.randn(B, H * G, Lq, D, generator=g).to(torch.bfloat16)
    table = np.arange(6).reshape(2, 3)
    kc = k.view(torch.uint8).numpy().reshape(B, H, 3, Pg, D).transpose(0, 2, 1, 3, 4).reshape(6, H, Pg, D)
    vc = v.view(torch.uint8).numpy().reshape(B, H, 3, Pg, D).transpose(0, 2, 1, 3, 4).reshape(6, H, Pg, D)
    one = np.full((6, H), 127, np.uint8)
    o, lse, _, _ = ref.attention(q.double().numpy(), kc, vc, one, one, table, [n, n], None, True, None, 0.125)
    mask = torch.arange(n)[None] <= torch.arange(n - Lq, n)[:, None]
    kk, vv = (t.double()[:, :, :n].repeat_interleave(G, 1) for t in (k, v))
    s = (q.double() @ kk.transpose(2, 3) * 0.125).masked_fill(~mask, -float("inf"))
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-12)
    np.testing.assert_allclose(o, (torch.softmax(s, -1) @ vv).numpy(), atol=1e-12)
