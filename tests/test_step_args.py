"""The verification step's entry points refuse bad arguments before they touch a device (CPU), and
the model that the GPU tests compare with holds to its own definitions."""
import ctypes

import numpy as np
import pytest

import suffix_match_drafter_amd as sfx
from tests import kv_model as M


def cache(**kw):
    c = dict(num_pages=4, page_size=64, kv_heads=2, head_dim=128, k=1024, v=2048, k_scale=4096,
             v_scale=8192)  # addresses that are checked, never read
    c.update(kw)
    return sfx._KvCache(*[c[f[0]] for f in sfx._KvCache._fields_])


P = ctypes.c_void_p(64)  # as above
BAD_CACHE = [(dict(num_pages=-1), "EINVAL"), (dict(kv_heads=0), "EINVAL"),
             (dict(head_dim=96), "EINVAL"), (dict(head_dim=0), "EINVAL"),
             (dict(page_size=16), "EINVAL"), (dict(page_size=48), "EINVAL"),
             (dict(page_size=0), "EINVAL"), (dict(page_size=4096), "EINVAL"),
             (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(k_scale=None), "EINVAL"),
             (dict(v_scale=None), "EINVAL"), (dict(k=1028), "EINVAL")]


def write(c, B=1, T=1, mp=2, table=P, start=P, count=None, k=P, v=P, ty=0, fn="sfx_kv_write"):
    return getattr(sfx.load(), fn)(ctypes.byref(c) if c else None, B, T, mp, table, start, count,
                                   k, None, v, None, ty, None)


def attend(c, B=1, T=1, H=4, mp=2, table=P, lens=P, q=P, out=P, ty=0, scale=0.1, window=0,
           sinks=0, ws=None, nws=0):
    return sfx.load().sfx_kv_attention(ctypes.byref(c) if c else None, B, T, H, mp, table, lens,
                                       None, q, None, out, ty, scale, window, sinks, ws, nws,
                                       None)


def verify(B=1, k=4, V=100000, logits=P, ty=0, draft=P, ua=P, us=P, out=P, na=P, ws=P, nws=1 << 20):
    return sfx.load().sfx_verify(B, k, V, logits, 0, 0, ty, None, draft, None, ua, us, out, na,
                                 ws, nws, None)


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_cache(kw, code):
    for rc in (write(cache(**kw)), write(cache(**kw), fn="sfx_kv_read"), attend(cache(**kw))):
        assert rc == getattr(sfx, code)
        assert len(sfx.load().sfx_last_error()) > 0


@pytest.mark.parametrize("fn", ["sfx_kv_write", "sfx_kv_read"])
def test_bad_move(fn):
    for kw in (dict(B=-1), dict(T=-1), dict(mp=-1), dict(table=None), dict(start=None),
               dict(k=None), dict(v=None), dict(ty=3), dict(ty=-1)):
        assert write(cache(), fn=fn, **kw) == sfx.EINVAL, kw
    assert write(None, fn=fn) == sfx.EINVAL
    assert write(cache(), mp=1 << 26, fn=fn) == sfx.ECAPACITY
    assert write(cache(), B=1 << 30, T=1 << 20, fn=fn) == sfx.ECAPACITY
    # nothing to do: nothing is looked at
    assert write(cache(), B=0, table=None, start=None, k=None, v=None, fn=fn) == sfx.OK
    assert write(cache(), T=0, table=None, start=None, k=None, v=None, fn=fn) == sfx.OK


def test_bad_attention():
    for kw in (dict(B=-1), dict(T=-1), dict(mp=-1), dict(H=3), dict(H=0), dict(table=None),
               dict(lens=None), dict(q=None), dict(out=None), dict(ty=2), dict(ty=5),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=-1), dict(sinks=-1),
               dict(out=ctypes.c_void_p(72))):
        assert attend(cache(), **kw) == sfx.EINVAL, kw
    assert attend(None) == sfx.EINVAL
    assert attend(cache(), mp=1 << 26) == sfx.ECAPACITY
    assert attend(cache(), B=1 << 20, T=1 << 20) == sfx.ECAPACITY
    assert attend(cache(), B=0, lens=None, q=None, out=None) == sfx.OK
    n = ctypes.c_size_t()
    L = sfx.load()
    c = cache()
    assert L.sfx_kv_attention_workspace_bytes(ctypes.byref(c), 1, 17, 4, 512, 0, 0,
                                              ctypes.byref(n)) == sfx.OK
    assert n.value > 0  # a long table alone on the card is split
    assert attend(c, T=17, mp=512) == sfx.EINVAL                       # no workspace
    assert attend(c, T=17, mp=512, ws=P, nws=n.value - 1) == sfx.EINVAL
    assert attend(c, T=17, mp=512, ws=ctypes.c_void_p(72), nws=n.value) == sfx.EINVAL
    assert L.sfx_kv_attention_workspace_bytes(ctypes.byref(c), 1, 17, 4, 512, 0, 0,
                                              None) == sfx.EINVAL


def test_bad_verify():
    for kw in (dict(B=-1), dict(k=-1), dict(k=33), dict(V=0), dict(V=-5), dict(V=(1 << 30) + 1),
               dict(logits=None), dict(ty=3), dict(draft=None), dict(ua=None), dict(us=None),
               dict(out=None), dict(na=None), dict(ws=None), dict(nws=8),
               dict(ws=ctypes.c_void_p(72))):
        assert verify(**kw) == sfx.EINVAL, kw
    assert verify(B=0, logits=None, us=None, ws=None) == sfx.OK
    n = ctypes.c_size_t()
    L = sfx.load()
    assert L.sfx_verify_workspace_bytes(4, 8, 1000, 0, None) == sfx.EINVAL
    assert L.sfx_verify_workspace_bytes(4, 33, 1000, 0, ctypes.byref(n)) == sfx.EINVAL
    assert L.sfx_verify_workspace_bytes(4, 8, 1000, 3, ctypes.byref(n)) == sfx.EINVAL
    assert L.sfx_verify_workspace_bytes(4, 8, 100000, 2, ctypes.byref(n)) == sfx.OK and n.value > 0


def test_python_refusals():
    import torch

    for a in ((1, 64, 2, 80), (1, 16, 2, 64), (1, 40, 2, 64), (-1, 64, 2, 64), (1, 64, 0, 64)):
        with pytest.raises(ValueError):
            sfx.KVCache(*a, device="cpu")
    c = sfx.KVCache(2, 64, 2, 64, device="cpu")
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        c.write(x, x, i[None], i)
    with pytest.raises(TypeError):
        c.attend(x, i[None], i)
    with pytest.raises(TypeError):
        c.read(i[None], i, None, 1)
    with pytest.raises(TypeError):
        sfx.verify(torch.zeros(1, 2, 5), i[None], i, torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(TypeError):
        sfx.KVCache(2, 64, 2, 64, buffers=(c.k, c.v, c.k_scale, c.v_scale))  # not on the GPU


# ------------------------------------------------------------------ the model
def test_model_codes():
    assert np.array_equal(M.encode(M.VALUES[:127]), np.arange(127))
    assert np.array_equal(M.encode(M.VALUES[128:255]), np.arange(128, 255))
    assert M.encode(1e9) == 126 and M.encode(-1e9) == 254 and M.encode(np.nan) & 127 == 127
    # halfway between neighbours: the even code; a hair to either side: the nearer one
    for c in range(126):
        mid = (M.VALUES[c] + M.VALUES[c + 1]) / 2
        assert M.encode(mid) == c + c % 2
        assert M.encode(np.nextafter(mid, 0)) == c
        assert M.encode(np.nextafter(mid, 1e9)) == c + 1
    for e in range(-30, 30):
        assert M.needed(448.0 * 2.0 ** e) == e
        assert M.needed(np.nextafter(448.0 * 2.0 ** e, np.inf)) == e + 1


def test_model_pack_is_a_permutation():
    c = M.Cache(2, 64, 3, 64)
    n = c.code["k"].size
    for name in "kv":
        idx = np.arange(n).reshape(c.shape)
        seen = np.zeros(n, np.int64)
        for shift in range(0, 16, 8):  # the position of every element, byte by byte
            c.code[name] = (idx >> shift & 255).astype(np.uint8)
            seen |= c.pack(name)[0].reshape(-1).astype(np.int64) << shift
        assert np.array_equal(np.sort(seen), np.arange(n))


def test_model_verification_keeps_the_distribution():
    """Over a grid of random numbers the first emitted token has the target's probabilities."""
    p = np.array([0.5, 0.2, 0.05, 0.25])
    logits = np.log(np.stack([p, p]))
    for d in range(4):
        got = np.zeros(4)
        grid = (np.arange(200) + 0.5) / 200
        for ua in grid:
            for us in grid:
                s, _ = M.verify(logits, np.array([d]), 1, np.array([ua]), us, 1.0)
                got[s[0]] += 1
        # each border of the two grids can misplace one line of 1 / 200
        assert np.abs(got / got.sum() - p).max() <= 2 / 200


def test_attention_scale_range():
    """A scale whose product with a block's power of two would not be a normal number is refused."""
    for scale in (2.0 ** 65, 2.0 ** -65, 1e-40, 3e38):
        assert attend(cache(), scale=scale) == sfx.EINVAL, scale
    for scale in (2.0 ** 64, 2.0 ** -64):
        assert attend(cache(), B=0, scale=scale) == sfx.OK, scale


def test_verification_weights_keep_their_bound():
    """The bound that the header states for sfx_verify's fp64 weights, over the kernel's arithmetic
    (a table of 2^(i / 256) and a cubic) with every operation rounded as there."""
    import os

    text = open(os.path.join(os.path.dirname(sfx.__file__), "..", "include", "sfx.h")).read()
    assert "within 2^-42 of exp" in text and "up to fp64 rounding" not in text
    z, magic = np.log(2.0) / 256, 1.5 * 2.0 ** 52
    wide = np.longdouble

    def fma(a, b, c):
        return np.float64(wide(a) * wide(b) + wide(c))

    rng = np.random.default_rng(0)
    for temp in (0.3, 0.7, 1.0, 1.7, 30.0):
        for reach in (1.0, 20.0, 700.0):
            d = -rng.uniform(0, reach, 20000) * temp
            k = np.float64(1.0 / temp) * (256 * np.float64(np.log2(np.e)))
            n = fma(d, k, magic) - magic
            f = fma(d, k, -n)
            n = n.astype(np.int64)
            t = np.ldexp(np.exp2((n & 255) / 256.0), (n >> 8).astype(np.int32))
            p = fma(f, fma(f, z ** 3 / 6, z * z / 2), z)
            got = fma(t, p * f, t)
            want = np.exp(wide(d) / wide(temp))
            assert np.abs(wide(got) / want - 1).max() <= 2.0 ** -42, (temp, reach)


def test_attention_leaves_matrix_results_to_the_compiler():
    """The wait states between a matrix instruction and a read of its result are put in by the
    compiler, which does not look into inline assembly: the attention has none with instructions."""
    import os
    import re

    path = os.path.join(os.path.dirname(sfx.__file__), "csrc", "kv_attention.hip")
    code = re.sub(r"//[^\n]*", "", open(path).read())
    texts = re.findall(r"\basm\b\s*(?:volatile\s*)?\(\s*\"([^\"]*)\"", code)
    assert len(texts) == len(re.findall(r"\b(?:__)?asm(?:__)?\b", code))
    assert all(t == "" for t in texts), texts


def test_launches_that_the_runtime_would_refuse():
    """A launch has at most 2^32 - 1 threads: larger calls are refused as too large, by the size
    queries too, and the largest ones that fit are not."""
    L = sfx.load()
    n = ctypes.c_size_t()

    def attention_bytes(B, T=1, heads=8, H=8, mp=2):
        c = cache(kv_heads=heads)
        return L.sfx_kv_attention_workspace_bytes(ctypes.byref(c), B, T, H, mp, 0, 0,
                                                  ctypes.byref(n))

    def verify_bytes(B, k, V):
        return L.sfx_verify_workspace_bytes(B, k, V, 0, ctypes.byref(n))

    # one workgroup of 256 threads per request and head
    assert attention_bytes((1 << 21) - 1) == sfx.OK
    assert attention_bytes(1 << 21) == sfx.ECAPACITY
    assert attend(cache(kv_heads=8), B=1 << 21, H=8) == sfx.ECAPACITY
    assert attention_bytes(1 << 21, T=0) == sfx.OK                     # no launch
    # 1024 threads a request; at larger vocabularies 256 a row and more
    assert verify_bytes((1 << 22) - 1, 0, 10) == verify_bytes((1 << 22) - 1, 3, 4096) == sfx.OK
    assert verify_bytes(1 << 22, 0, 10) == sfx.ECAPACITY
    assert verify(B=1 << 22, k=0, V=10) == sfx.ECAPACITY
    assert verify_bytes(508400, 32, 5000) == sfx.OK
    assert verify_bytes(508401, 32, 5000) == sfx.ECAPACITY
    # one wavefront per request, block, tensor and head
    for fn in ("sfx_kv_write", "sfx_kv_read"):
        assert write(cache(), B=1 << 24, fn=fn) == sfx.ECAPACITY
        assert write(cache(kv_heads=2 ** 31 - 1), B=2 ** 31 - 1, T=2 ** 31 - 1,
                     fn=fn) == sfx.ECAPACITY
    # products past 64 bits
    assert attention_bytes(2 ** 31 - 1, T=1, heads=2 ** 31 - 1, H=2 ** 31 - 1) == sfx.ECAPACITY


def test_sizes_past_32_bits_are_refused():
    """They would reach the library modulo 2^32."""
    for pages, heads in ((2 ** 32 + 1, 1), (0, 2 ** 32 + 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            sfx.KVCache(pages, 64, heads, 64, device="meta")


def test_cache_keeps_its_buffers():
    """The library reads the memory that the cache was made with: another tensor in its place would
    be ignored, so it is refused."""
    import torch

    c = sfx.KVCache(2, 64, 1, 64, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale", "num_pages", "page_size", "kv_heads", "head_dim",
                 "device"):
        was = getattr(c, name)
        with pytest.raises(AttributeError, match=name):
            setattr(c, name, was.clone() if isinstance(was, torch.Tensor) else was)
        assert getattr(c, name) is was
    c.k.fill_(7)
    c.owner = "a request"  # a caller's own attribute
    assert c._c.k == c.k.data_ptr() and int(c.k.sum()) == 7 * c.k.numel()


def test_gradients_are_refused():
    import torch

    x = torch.zeros(1, 1, 2, 64, requires_grad=True)
    with pytest.raises(RuntimeError, match="q requires grad"):
        sfx._heads(x, "q", 2, 64, -1)
    with torch.no_grad():
        assert sfx._heads(x, "q", 2, 64, -1) == x.shape
    assert sfx._heads(x.detach(), "q", 2, 64, -1) == x.shape
