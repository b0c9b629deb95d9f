"""The 8-bit KV cache's write and read against the model in 64 bits (tests/kv_model.py).  Block
scales are powers of two, so every stored code and scale is compared exactly."""
import numpy as np
import pytest

from tests import kv_model as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import suffix_match_drafter_amd as sfx

    sfx.load()
    return sfx


def dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(x):
    return dev(np.asarray(x, np.int32))


TYPES = ("bfloat16", "float16", "float32")


def inputs(rng, shape, dtype, scale=1.0):
    """Values of `dtype` and their float64 equals: several magnitudes, zeros, exact ties."""
    import torch

    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, size=shape[:-1] + (1,))) * scale
    x[rng.random(shape) < 0.05] = 0.0
    t = torch.from_numpy(x).to(getattr(torch, dtype))
    return t.cuda(), t.double().numpy()


def check(cache, model):
    import torch

    torch.cuda.synchronize()
    for name in "kv":
        code, scale = model.pack(name)
        got = getattr(cache, name).view(torch.uint8).cpu().numpy()
        gs = getattr(cache, name + "_scale").cpu().numpy()
        # +-NaN and +-0 are compared as values
        a, b = M.VALUES[got], M.VALUES[code]
        bad = ~((a == b) | (np.isnan(a) & np.isnan(b)))
        assert not bad.any(), (name, np.argwhere(bad)[:5], a[bad][:5], b[bad][:5])
        assert np.array_equal(np.where(gs == 0, np.float32(2.0 ** M.E_LO), gs), scale), name


def write(cache, model, k, v, table, start, count):
    """Both sides; k and v are (tensor, float64)."""
    cache.write(k[0], v[0], i32(table), i32(start), None if count is None else i32(count))
    B, T = k[1].shape[:2]
    for b in range(B):
        n = T if count is None else count[b]
        for name, x in (("k", k), ("v", v)):
            model.write(name, x[1][b], table[b], start[b], n)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_then_tokens(S, dtype, dim):
    """A ragged prompt, then drafts of several lengths over ends of blocks and pages, some of
    them written again from an earlier position (rejected drafts), with growing magnitudes."""
    rng = np.random.default_rng(dim + len(dtype))
    B, H, page, pages = 3, 2, 64, 14
    cache, model = S.KVCache(pages, page, H, dim), M.Cache(pages, page, H, dim)
    table = rng.permutation(pages)[:12].reshape(B, 4)
    k, v = inputs(rng, (B, 70, H, dim), dtype), inputs(rng, (B, 70, H, dim), dtype)
    write(cache, model, k, v, table, [0, 0, 0], [70, 33, 1])
    check(cache, model)
    at = [70, 33, 1]
    for step, T in enumerate((1, 5, 17, 33, 2)):
        k, v = (inputs(rng, (B, T, H, dim), dtype, 2.0 ** step) for _ in range(2))
        write(cache, model, k, v, table, at, [T, max(0, T - 1), T])
        check(cache, model)
        at = [a + int(x) for a, x in zip(at, rng.integers(0, T + 1, size=B))]


@pytest.mark.parametrize("dtype", TYPES)
def test_extremes(S, dtype):
    """Zeros, the type's largest and smallest values, infinities, NaN, blocks of one magnitude at
    the border between two scales, magnitudes past the exponents' range."""
    import torch

    H, dim, page = 1, 64, 32
    t = getattr(torch, dtype)
    fi = torch.finfo(t)
    rows = [torch.zeros(32, dim), torch.full((32, dim), fi.max), torch.full((32, dim), fi.tiny),
            torch.full((32, dim), -448.0), torch.full((32, dim), 449.0 if t != torch.bfloat16
                                                      else 450.0),
            torch.full((32, dim), 2.0 ** -43 if t != torch.float16 else 2.0 ** -24)]
    x = torch.randn(32, dim, generator=torch.Generator().manual_seed(1))
    rows.append(x.clone())
    rows[-1][3, 5], rows[-1][4, 6], rows[-1][31, 63], rows[-1][0, 0] = (
        float("inf"), -float("inf"), float("nan"), float("-nan"))
    rows.append(torch.full((32, dim), float("nan")))
    rows.append(torch.full((32, dim), float("inf")))
    if t != torch.float16:
        rows += [x * 2.0 ** 40, x * 2.0 ** -45, x * 2.0 ** 120]
    data = torch.cat(rows)[None, :, None].to(t)
    n = data.shape[1]
    cache, model = S.KVCache(n // 32, page, H, dim), M.Cache(n // 32, page, H, dim)
    table = np.arange(n // 32)[::-1][None]
    pair = (data.cuda(), data.double().numpy())
    write(cache, model, pair, pair, table, [0], None)
    check(cache, model)
    # and appended behind live tokens: the blocks' scales grow or stay
    cache2, model2 = S.KVCache(n // 32, page, H, dim), M.Cache(n // 32, page, H, dim)
    first = inputs(np.random.default_rng(0), (1, n, H, dim), dtype)
    write(cache2, model2, first, first, table, [0], None)
    for a in range(0, n, 32):
        one = (pair[0][:, a:a + 16].contiguous(), pair[1][:, a:a + 16])
        write(cache2, model2, one, one, table, [a + 9], None)
    check(cache2, model2)


def test_unmapped_and_clamped(S):
    """Bad page ids, starts and counts write nothing and read as zero."""
    import torch

    rng = np.random.default_rng(5)
    H, dim, page, pages = 3, 64, 32, 6
    cache, model = S.KVCache(pages, page, H, dim), M.Cache(pages, page, H, dim)
    table = np.array([[0, -1, 2], [pages, 4, 2 ** 31 - 1], [5, 3, 1], [-2 ** 31, -1, -1]])
    B, T = 4, 90
    k, v = (inputs(rng, (B, T, H, dim), "float32") for _ in range(2))
    write(cache, model, k, v, table, [3, 0, -1, 0], [90, 1000, 90, 90])
    check(cache, model)
    write(cache, model, k, v, table, [0, 80, 7, 2 ** 31 - 1], [0, 90, -5, 90])
    check(cache, model)
    start, count = [3, 0, 50, -7], [80, 200, 30, 5]
    got = cache.read(i32(table), i32(start), i32(count), T, torch.float32)
    for name, g in zip("kv", got):
        g = g.cpu().numpy()
        for b in range(B):
            want = np.zeros((T, H, dim))
            if start[b] >= 0:
                n = min(count[b], T)
                vals, _ = model.values(name, table[b], start[b] + n)
                want[:n] = vals[start[b]:start[b] + n]
            assert np.array_equal(g[b], want.astype(np.float32)), (name, b)
    far = cache.read(i32(table), i32([2 ** 31 - 1] * 4), None, 40, torch.float32)
    assert not any(x.any().item() for x in far)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_read_back(S, dtype, dim):
    """Whatever was stored comes back rounded once; spans start and end inside blocks."""
    import torch

    rng = np.random.default_rng(dim)
    B, H, page, pages = 3, 5, 96, 9
    cache, model = S.KVCache(pages, page, H, dim), M.Cache(pages, page, H, dim)
    table = rng.permutation(pages).reshape(B, 3)
    k, v = (inputs(rng, (B, 280, H, dim), "float32") for _ in range(2))
    write(cache, model, k, v, table, [0, 0, 0], [280, 97, 31])
    for T, start, count in ((1, [0, 96, 30], [1, 1, 1]), (45, [10, 60, 0], [45, 37, 0]),
                            (280, [0, 0, 0], [280, 97, 31]), (33, [31, 32, 0], None)):
        got = cache.read(i32(table), i32(start), None if count is None else i32(count), T,
                         getattr(torch, dtype))
        for name, g in zip("kv", got):
            assert g.dtype == getattr(torch, dtype)
            for b in range(B):
                n = T if count is None else count[b]
                vals, _ = model.values(name, table[b], 288)
                want = torch.zeros((T, H, dim), dtype=torch.float64)
                want[:n] = torch.from_numpy(vals[start[b]:start[b] + n])
                assert torch.equal(g[b].cpu(), want.to(g.dtype)), (name, b, T)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_strides(S, dtype):
    """Slices of one fused projection at odd offsets, batches and heads of any stride."""
    import torch

    rng = np.random.default_rng(9)
    B, T, H, dim, page = 2, 37, 2, 64, 32
    t = getattr(torch, dtype)
    fused = torch.from_numpy(rng.standard_normal((B, T, 3 + 2 * H * dim + 4))).to(t).cuda()
    k = fused[:, :, 3:3 + H * dim].view(B, T, H, dim)
    v = fused[:, :, 3 + H * dim:3 + 2 * H * dim].view(B, T, H, dim)
    kt = torch.from_numpy(rng.standard_normal((H, T, B, dim))).to(t).cuda().permute(2, 1, 0, 3)
    for a, b in ((k, v), (kt, v)):
        cache, model = S.KVCache(6, page, H, dim), M.Cache(6, page, H, dim)
        table = np.array([[5, 0, 3], [1, 2, 4]])
        write(cache, model, (a, a.double().cpu().numpy()), (b, b.double().cpu().numpy()), table,
              [1, 20], None)
        check(cache, model)
        out = torch.full((B, T, 5 + 2 * H * dim), 7.0, dtype=t, device="cuda")
        ko = out[:, :, 3:3 + H * dim].view(B, T, H, dim)
        vo = out[:, :, 3 + H * dim:3 + 2 * H * dim].view(B, T, H, dim)
        kd, vd = cache.read(i32(table), i32([1, 20]), None, T, t)
        cache.read(i32(table), i32([1, 20]), None, T, t, k=ko, v=vo)
        assert torch.equal(ko, kd) and torch.equal(vo, vd)
        assert (out[:, :, :3] == 7).all() and (out[:, :, 3 + 2 * H * dim:] == 7).all()


def test_empty_calls(S):
    import torch

    cache = S.KVCache(0, 32, 2, 64)
    x = torch.randn(2, 3, 2, 64, device="cuda")
    cache.write(x, x, i32([[0], [-1]]), i32([0, 0]))
    assert not cache.read(i32([[0], [-1]]), i32([0, 0]), None, 3)[0].any().item()
    cache = S.KVCache(2, 32, 2, 64)
    none = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    cache.write(x, x, none, i32([0, 0]))
    assert not cache.k.any().item()
    assert not cache.read(none, i32([0, 0]), None, 3)[1].any().item()
    cache.write(x[:, :0], x[:, :0], i32([[0], [1]]), i32([0, 0]))
    cache.write(x[:0], x[:0], i32([[0], [1]])[:0], i32([]))
    assert cache.read(i32([[0], [1]]), i32([0, 0]), None, 0)[0].shape == (2, 0, 2, 64)
    assert not cache.k.any().item()


def test_offsets_past_32_bits(S):
    """A page whose codes lie past 4 GiB."""
    import torch

    H, dim, page = 8, 128, 2048
    pages = (1 << 32) // (H * dim * page) + 3
    cache = S.KVCache(pages, page, H, dim)
    rng = np.random.default_rng(3)
    k, v = (inputs(rng, (1, 40, H, dim), "bfloat16") for _ in range(2))
    last = pages - 1
    cache.write(k[0], v[0], i32([[last]]), i32([2001]))
    model = M.Cache(1, page, H, dim)
    for name, x in (("k", k), ("v", v)):
        model.write(name, x[1][0], [0], 2001, 40)
    got = cache.read(i32([[last]]), i32([2001]), None, 40, torch.float32)
    for name, g in zip("kv", got):
        want, _ = model.values(name, [0], 2041)
        assert np.array_equal(g[0].cpu().numpy(), want[2001:].astype(np.float32))
    assert not cache.k[:last].any().item()


def test_graph_and_stream(S):
    """Captured write and read, replayed between eager work; and a stream of the caller's."""
    import torch

    rng = np.random.default_rng(4)
    B, T, H, dim, page = 2, 5, 2, 64, 32
    cache, model = S.KVCache(4, page, H, dim), M.Cache(4, page, H, dim)
    table = np.array([[0, 1], [2, 3]])
    ti, st = i32(table), i32([0, 0])
    k, v = (inputs(rng, (B, T, H, dim), "bfloat16") for _ in range(2))
    kb, vb = k[0].clone(), v[0].clone()
    ko, vo = torch.empty_like(kb), torch.empty_like(vb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.write(kb, vb, ti, st, stream=s)
        cache.read(ti, st, None, T, k=ko, v=vo, stream=s)
    for step in range(4):
        k, v = (inputs(rng, (B, T, H, dim), "bfloat16", 2.0 ** step) for _ in range(2))
        kb.copy_(k[0])
        vb.copy_(v[0])
        st.fill_(step * T)
        g.replay()
        for b in range(B):
            model.write("k", k[1][b], table[b], step * T, T)
            model.write("v", v[1][b], table[b], step * T, T)
        check(cache, model)
        for name, o in (("k", ko), ("v", vo)):
            want = np.stack([model.values(name, table[b], 64)[0][step * T:step * T + T]
                             for b in range(B)])
            assert np.array_equal(o.double().cpu().numpy(), want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    k, v = (inputs(rng, (B, T, H, dim), "float16") for _ in range(2))
    cache.write(k[0], v[0], ti, i32([33, 40]), stream=other)
    other.synchronize()
    for b, a in enumerate((33, 40)):
        model.write("k", k[1][b], table[b], a, T)
        model.write("v", v[1][b], table[b], a, T)
    check(cache, model)


def test_sizes_past_32_bits_are_refused(S):
    """2^32 + 1 tokens (of one token's memory) would reach the library as 1."""
    import torch

    cache = S.KVCache(1, 32, 1, 64)
    table, start, far = i32([[0]]), i32([0]), 2 ** 32 + 1
    x = torch.ones((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda").expand(1, far, 1, 64)
    for call in (lambda: cache.write(x, x, table, start, i32([5])),
                 lambda: cache.read(table, start, None, far, k=x, v=x),
                 lambda: cache.attend(x, table, start)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert not cache.k.any().item()
