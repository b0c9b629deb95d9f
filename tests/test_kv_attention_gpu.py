"""Attention over the 8-bit cache against the model in 64 bits, over the values that the cache
holds.

Tolerance of one output o = sum p v, from the kernel's roundings:
  the result's own rounding, eps/2 of |o|;
  each weight p rounded to fp16, 2^-11 of it, and below 2^-22 of the largest weight to a multiple
  of 2^-33 of it at worst, once per token;
  a score's fp32 error: (dim + 8) 2^-24 of sum |q||k| scale plus its own size, twice (numerator
  and denominator), as a relative error of the weights;
  fp32 sums: one rounding of 2^-23 per 32 tokens, 64 more in and after the matrix product;
all but the first in units of A = sum p |v|."""
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


def filled(S, rng, pages, page, heads, dim, spread=2):
    """A cache of random codes without NaN, block exponents within `spread` of -8."""
    model = M.Cache(pages, page, heads, dim)
    for n in "kv":
        x = rng.standard_normal(model.shape) * 60
        model.code[n] = M.encode(x)
        model.exp[n] = rng.integers(-8 - spread, -7 + spread, size=model.exp[n].shape)
    return upload(S, model), model


def upload(S, model):
    P, H, page, d = model.shape
    bufs = [None] * 4
    for i, n in enumerate("kv"):
        c, s = model.pack(n)
        bufs[i], bufs[2 + i] = dev(c), dev(s)
    return S.KVCache(P, page, H, d, buffers=tuple(bufs))


def compare(got, model, q, table, lens, qlens, scale, window, sinks):
    import torch

    eps = torch.finfo(got.dtype).eps / 2
    dim = model.shape[3]
    got = got.double().cpu().numpy()
    q = q.double().cpu().numpy()
    for b in range(q.shape[0]):
        n = q.shape[1] if qlens is None else qlens[b]
        ref, mag, dots = M.attention(model, q[b], table[b], lens[b], n, scale, window, sinks)
        L = max(lens[b], 1)
        rel = 2.0 ** -11 + 2 * (dim + 8) * 2.0 ** -24 * (dots + 1)[:, :, None] + \
            (L / 32 + 64) * 2.0 ** -23
        vmax = mag.max() if mag.size else 0.0
        tol = eps * np.abs(ref) + mag * rel + L * 2.0 ** -33 * max(
            vmax, np.abs(M.VALUES[:127]).max() * 2.0 ** int(model.exp["v"].max()))
        assert np.isfinite(got[b]).all(), b
        err = np.abs(got[b] - ref)
        assert (err <= tol).all(), (b, np.argwhere(err > tol)[:4], err.max(), tol.min(),
                                    got[b][err > tol][:4], ref[err > tol][:4])


CASES = [
    # B, T, heads, group, dim, page, lens, q_lens, window, sinks
    (2, 1, 1, 1, 64, 32, [1, 0], None, 0, 0),
    (3, 1, 2, 4, 128, 64, [33, 1000, 31], None, 0, 0),
    (2, 5, 2, 3, 64, 96, [5, 3], [5, 5], 0, 0),          # a row before the first token
    (3, 9, 1, 8, 128, 32, [9, 64, 200], [0, 9, 4], 0, 0),  # one 16-row tile to five
    (2, 17, 2, 8, 128, 64, [17, 777], [17, 16], 0, 0),
    (1, 33, 1, 5, 256, 128, [500], [33], 0, 0),
    (2, 3, 2, 16, 256, 64, [3, 260], [2, 3], 0, 0),
    (1, 70, 1, 1, 64, 32, [300], [70], 0, 0),
    (2, 4, 1, 2, 128, 64, [700, 90], [4, 3], 1, 0),      # sees itself alone
    (2, 4, 1, 2, 128, 64, [700, 90], [4, 3], 100, 0),
    (2, 4, 1, 2, 128, 64, [700, 90], [4, 3], 33, 4),
    (2, 17, 1, 4, 64, 32, [900, 40], [17, 17], 64, 100),  # sinks of several tiles
    (1, 2, 2, 2, 64, 32, [640], [2], 5, 1000),            # sinks past the window: everything
    (1, 1, 8, 1, 128, 2048, [4000], None, 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_model(S, case, dtype):
    import torch

    B, T, heads, group, dim, page, lens, qlens, window, sinks = case
    rng = np.random.default_rng(B * 1000 + T * 10 + dim)
    width = max(max(lens) // page + 2, 2)
    cache, model = filled(S, rng, B * width, page, heads, dim)
    table = rng.permutation(B * width).reshape(B, width)
    q = dev(rng.standard_normal((B, T, heads * group, dim))).to(getattr(torch, dtype))
    out = cache.attend(q, i32(table), i32(lens), None if qlens is None else i32(qlens),
                       window=window, sinks=sinks)
    compare(out, model, q, table, lens, qlens, dim ** -0.5, window, sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [16, 17, 33, 49, 65, 68, 81, 97, 119, 136, 150])
def test_row_chunks(S, dim, rows):
    """Every way of cutting a head's rows into chunks, split and not, with fewer live rows than
    there is room for."""
    import torch

    rng = np.random.default_rng(rows)
    page, group = 64, next(g for g in (17, 7, 4, 3, 2, 1) if rows % g == 0)
    T = rows // group
    for lens, width in (([90, 3], 3), ([2500, 700], 40)):
        cache, model = filled(S, rng, 2 * width, page, 1, dim)
        table = rng.permutation(2 * width).reshape(2, width)
        q = dev(rng.standard_normal((2, T, group, dim))).to(torch.bfloat16)
        qlens = [T, max(0, T - 2)]
        out = cache.attend(q, i32(table), i32(lens), i32(qlens))
        compare(out, model, q, table, lens, qlens, dim ** -0.5, 0, 0)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_long_and_split(S, dtype):
    """Long requests beside short ones: several splits, some of them empty."""
    import torch

    rng = np.random.default_rng(11)
    B, T, heads, group, dim, page, width = 3, 3, 1, 2, 64, 256, 48
    cache, model = filled(S, rng, B * width, page, heads, dim)
    table = rng.permutation(B * width).reshape(B, width)
    q = dev(2 * rng.standard_normal((B, T, heads * group, dim))).to(getattr(torch, dtype))
    for lens in ([12000, 1, 600], [12288, 0, 5000]):
        out = cache.attend(q, i32(table), i32(lens))
        compare(out, model, q, table, lens, None, dim ** -0.5, 0, 0)


def test_exponents_far_apart(S):
    """Neighbouring blocks whose scales differ by up to 2^60: the running references move."""
    import torch

    rng = np.random.default_rng(12)
    heads, dim, page, width = 2, 64, 32, 40
    for lo, hi in ((-32, 32), (-12, 8)):
        model = M.Cache(width, page, heads, dim)
        for n in "kv":
            model.code[n] = M.encode(rng.standard_normal(model.shape) * 100)
            model.exp[n] = rng.integers(lo, hi, size=model.exp[n].shape)
        model.exp["k"] = rng.integers(-32, -8, size=model.exp["k"].shape)  # scores stay modest
        cache = upload(S, model)
        table = rng.permutation(width)[None]
        for dtype in (torch.float16, torch.bfloat16):
            if dtype == torch.float16:
                model.exp["v"] = np.clip(model.exp["v"], -32, 5)  # results within fp16
                cache = upload(S, model)
            q = dev(rng.standard_normal((1, 6, heads * 3, dim))).to(dtype)
            lens = [width * page - 7]
            out = cache.attend(q, i32(table), i32(lens), scale=0.7)
            compare(out, model, q, table, lens, None, float(np.float32(0.7)), 0, 0)


def test_peaked_and_growing_scores(S):
    """Scores that grow along the sequence move the running maximum all the time; a late token
    that outweighs all others; scores hundreds apart."""
    import torch

    rng = np.random.default_rng(13)
    heads, dim, page, width = 1, 64, 32, 20
    L = width * page
    model = M.Cache(width, page, heads, dim)
    base = rng.standard_normal(dim)
    for n in "kv":
        model.code[n] = M.encode(rng.standard_normal(model.shape) * 30)
        model.exp[n][:] = -5
    grow = np.linspace(0, 300, L)[:, None] * base / np.abs(base).max()
    model.code["k"] = M.encode(grow.reshape(width, page, heads, dim).transpose(0, 2, 1, 3))
    table = np.arange(width)[None]
    for sign in (1.0, -1.0):
        cache = upload(S, model)
        q = dev(sign * np.tile(base, (1, 2, 3, 1)) * rng.uniform(0.5, 2, (1, 2, 3, 1)))
        for dtype in (torch.bfloat16, torch.float16):
            out = cache.attend(q.to(dtype), i32(table), i32([L]), scale=0.5)
            compare(out, model, q.to(dtype), table, [L], None, 0.5, 0, 0)


def test_nan_in_unseen_places(S):
    """NaN codes in tokens that a row does not see (later drafts, past the end, before the
    window, unmapped) leave it alone; in tokens that it sees they make it NaN."""
    import torch

    rng = np.random.default_rng(14)
    heads, dim, page, width, T, G = 2, 128, 32, 8, 6, 3
    cache, model = filled(S, rng, width, page, heads, dim)
    table = np.array([[3, 1, 0, 2, 5, 4, 7, 6]])
    L = 150
    clean = {n: model.code[n].copy() for n in "kv"}

    def poison(name, tok, d):
        model.code[name][table[0][tok // page], :, tok % page, d] = 127

    q = dev(rng.standard_normal((1, T, heads * G, dim))).to(torch.float16)
    for name, d in (("v", 5), ("k", 70), ("v", slice(None))):
        for n in "kv":
            model.code[n] = clean[n].copy()
        for tok in (L, L + 1, 159, 165, 20, 41, L - 2):  # past the end; before the window; draft 4
            poison(name, tok, d)
        out = upload(S, model).attend(q, i32(table), i32([L]), window=60, sinks=4)
        good = M.Cache(*[model.shape[i] for i in (0, 2, 1, 3)])
        good.code, good.exp = clean, model.exp
        got = out.float().cpu()
        # row t stands at 144 + t: rows 4 and 5 see token 148
        hit = got[0, 4:]
        want_nan = hit if name == "k" else hit[..., d]
        assert torch.isnan(want_nan).all()
        if name == "v" and d == 5:
            assert torch.isfinite(hit[..., :5]).all() and torch.isfinite(hit[..., 6:]).all()
        compare(out[:, :4], good, q[:, :4], table, [L - 2], None, dim ** -0.5, 60, 4)


def test_nan_in_fully_seen_tiles(S):
    import torch

    rng = np.random.default_rng(15)
    heads, dim, page, width = 1, 64, 32, 6
    cache, model = filled(S, rng, width, page, heads, dim)
    model.code["v"][2, :, 7, 9] = 255
    table = np.arange(width)[None]
    q = dev(rng.standard_normal((1, 2, 2, dim))).to(torch.bfloat16)
    out = upload(S, model).attend(q, i32(table), i32([190])).float().cpu()
    bad = torch.isnan(out)
    assert bad[..., 9].all() and bad.sum() == 4
    out = upload(S, model).attend(q, i32(table), i32([64])).float()  # not that far
    assert torch.isfinite(out).all()


def test_unmapped_pages(S):
    """Tokens of unmapped pages are not seen; a row with nothing else is zero."""
    import torch

    rng = np.random.default_rng(16)
    heads, dim, page = 2, 64, 32
    cache, model = filled(S, rng, 4, page, heads, dim)
    table = np.array([[0, -1, 2], [4, -7, 2 ** 31 - 1], [3, 1, -2 ** 31]])
    q = dev(rng.standard_normal((3, 2, 4, dim))).to(torch.bfloat16)
    lens = [96, 96, 2000]  # the last is clamped to the table
    out = cache.attend(q, i32(table), i32(lens))
    compare(out, model, q, table, [96, 96, 96], None, dim ** -0.5, 0, 0)
    assert not out[1].any().item()
    none = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    assert not cache.attend(q, none, i32(lens)).any().item()
    assert not S.KVCache(0, 32, heads, dim).attend(q, i32(table), i32(lens)).any().item()


def test_bad_lengths_are_clamped(S):
    import torch

    rng = np.random.default_rng(17)
    heads, dim, page = 1, 64, 32
    cache, model = filled(S, rng, 4, page, heads, dim)
    table = np.array([[0, 1], [2, 3], [1, 2]])
    q = dev(rng.standard_normal((3, 3, 2, dim))).to(torch.float16)
    out = cache.attend(q, i32(table), i32([-5, 2 ** 31 - 1, 40]), i32([3, 99, -1]))
    compare(out, model, q, table, [0, 64, 40], [3, 3, 0], dim ** -0.5, 0, 0)
    assert not out[0].any().item() and not out[2].any().item()


def test_garbage_in_unused_memory(S):
    """Memory that was never written (NaN codes, wild scales) past the lengths changes nothing."""
    import torch

    rng = np.random.default_rng(18)
    heads, dim, page = 2, 128, 64
    cache, model = filled(S, rng, 6, page, heads, dim)
    table = np.array([[0, 1, 2], [3, 4, 5]])
    q = dev(rng.standard_normal((2, 3, 8, dim))).to(torch.bfloat16)
    lens = [65, 100]
    want = cache.attend(q, i32(table), i32(lens))
    for b, L in enumerate(lens):
        for pi in range(3):
            for n in "kv":
                live = max(0, min(64, L - pi * 64))
                model.code[n][table[b][pi], :, live:] = 255
    bad = upload(S, model)
    for s in (bad.k_scale, bad.v_scale):
        for b, L in enumerate(lens):
            blocks = s[i32(table[b]).long()].transpose(0, 1).reshape(heads, -1).clone()
            blocks[:, (L + 31) // 32:] = float("nan")
            s[i32(table[b]).long()] = blocks.view(heads, 3, 2).transpose(0, 1)
    assert torch.equal(bad.attend(q, i32(table), i32(lens)), want)


def test_strided_queries(S):
    import torch

    rng = np.random.default_rng(19)
    B, T, heads, group, dim = 2, 5, 2, 2, 64
    cache, model = filled(S, rng, 8, 32, heads, dim)
    table = rng.permutation(8).reshape(2, 4)
    fused = dev(rng.standard_normal((B, T, 3 + heads * group * dim + 2))).to(torch.bfloat16)
    q = fused[:, :, 3:3 + heads * group * dim].view(B, T, heads * group, dim)
    q2 = dev(rng.standard_normal((heads * group, B, T, dim))).to(torch.float16).permute(1, 2, 0,
                                                                                        3)
    for x in (q, q2):
        out = torch.full((B, T, heads * group, dim), 3.0, dtype=x.dtype, device="cuda")
        got = cache.attend(x, i32(table), i32([100, 7]), out=out)
        assert got is out
        compare(out, model, x, table, [100, 7], None, dim ** -0.5, 0, 0)
    assert cache.attend(q[:, :0], i32(table), i32([100, 7])).shape == (B, 0, 4, dim)
    assert cache.attend(q[:0], i32(table)[:0], i32([])).shape == (0, T, 4, dim)


def test_offsets_past_32_bits(S):
    """Pages whose codes lie past 4 GiB."""
    import torch

    rng = np.random.default_rng(20)
    heads, dim, page = 8, 128, 2048
    pages = (1 << 32) // (heads * dim * page) + 3
    cache = S.KVCache(pages, page, heads, dim)
    model = M.Cache(1, page, heads, dim)
    k, v = (rng.standard_normal((1, 300, heads, dim)) for _ in range(2))
    k, v = (dev(x).to(torch.bfloat16) for x in (k, v))
    table = [[pages - 1]]
    cache.write(k, v, i32(table), i32([0]))
    for n, x in (("k", k), ("v", v)):
        model.write(n, x[0].double().cpu().numpy(), [0], 0, 300)
    q = dev(rng.standard_normal((1, 2, heads, dim))).to(torch.bfloat16)
    out = cache.attend(q, i32(table), i32([300]))
    compare(out, model, q, [[0]], [300], None, dim ** -0.5, 0, 0)


def test_graph_stream_and_repeat(S):
    """Captured calls (split and not) replayed between eager work equal eager ones bit for bit;
    so does a stream of the caller's, and a second call."""
    import torch

    rng = np.random.default_rng(21)
    heads, dim, page, width = 2, 64, 64, 64
    cache, model = filled(S, rng, 2 * width, page, heads, dim)
    table = i32(rng.permutation(2 * width).reshape(2, width))
    q = dev(rng.standard_normal((2, 4, 8, dim))).to(torch.bfloat16)
    lens, ql = i32([4000, 50]), i32([4, 3])
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.attend(q, table, lens, ql, out=out, stream=s)
    for step in range(4):
        q.copy_(dev(rng.standard_normal((2, 4, 8, dim))))
        lens.copy_(i32([4000 - 900 * step, 50 + 700 * step]))
        out.fill_(5.0)
        want = cache.attend(q, table, lens, ql)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
        assert torch.equal(cache.attend(q, table, lens, ql), want)
        s.wait_stream(torch.cuda.current_stream())
        mine = cache.attend(q, table, lens, ql, stream=s)
        s.synchronize()
        assert torch.equal(mine, want)
    compare(want, model, q, table.cpu().numpy(), lens.cpu().tolist(), [4, 3], dim ** -0.5, 0, 0)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("power", [16, 24, 27, 28, 30, 40, 60, 100])
def test_very_large_scores(S, dtype, power):
    """Scores of about +-2^power, where a step of fp32 passes the softmax's whole range: the token
    that leads by more than the scores' error has all the weight (its own is rounded by 2^-11)."""
    import torch

    rng = np.random.default_rng(power)
    heads, dim, page, T = 1, 64, 64, 3
    dt = getattr(torch, dtype)
    for L, width in ((70, 2), (2500, 40)):
        model = M.Cache(width, page, heads, dim)
        for n in "kv":
            model.code[n] = M.encode(np.abs(rng.standard_normal(model.shape)) * 60)
            model.exp[n][:] = -8
        # one token far ahead, one far behind
        model.code["k"][0, :, 5] = M.encode(np.full((heads, dim), 400.0))
        model.code["k"][1, :, 3] = M.encode(np.full((heads, dim), 2.0 ** -5))
        # the largest |sum q k| is about 2^15 times the units of q and of the keys
        unit = max(-8, min(31, power - 20)) if dtype == "float16" else -8
        model.exp["k"][:] = unit
        big, scale = (5, 2.0 ** (power - 21 - unit)) if dtype == "float16" else \
            (power - 16 - unit, 1.0)
        cache = upload(S, model)
        table = np.arange(width)[None]
        x = np.abs(rng.standard_normal((1, T, 4, dim))) + 0.5
        x[:, :, 1::2] *= -1
        q = dev(x * 2.0 ** big).to(dt)
        out = cache.attend(q, i32(table), i32([L]), scale=scale).double().cpu().numpy()
        keys, values = (model.values(n, table[0], L)[0][:, 0] for n in "kv")
        for t in range(T):
            see = L - T + t + 1
            for h in range(4):
                row = q[0, t, h].double().cpu().numpy()
                s = keys[:see] @ row * scale * np.log2(np.e)
                err = 2 * (dim + 8) * 2.0 ** -24 * (np.abs(keys[:see]) @ np.abs(row)).max() * \
                    scale * np.log2(np.e)
                order = np.argsort(s)
                assert s[order[-1]] - s[order[-2]] > 64 + err
                assert 2.0 ** (power - 12) < np.abs(s).max() < 2.0 ** (power + 6)
                want = values[order[-1]]
                tol = (torch.finfo(dt).eps / 2 + 2.0 ** -11 + 2.0 ** -20) * np.abs(want)
                assert (np.abs(out[0, t, h] - want) <= tol).all(), (L, t, h)


def test_window_past_32_bits_is_refused(S):
    import torch

    cache = S.KVCache(1, 32, 1, 64)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.float16, device="cuda")
    for kw in (dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(sinks=2 ** 32), dict(sinks=-1)):
        with pytest.raises(ValueError):
            cache.attend(q, i32([[0]]), i32([0]), **kw)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("power", [8, 16, 18, 20, 24, 28, 34])
@pytest.mark.parametrize("counts", [(48, 16, 0, 5), (1, 300, 7, 0), (3, 1, 1, 1)], ids=str)
def test_equal_large_scores(S, dtype, power, counts):
    """Tokens of one key, whose scores of +-2^power are equal to the last bit, share the softmax
    equally however they are spread over a long request's splits; all others are far behind.  So
    the scores' error does not count: the result's own rounding, the weights' 2^-11 and the fp32
    sums do."""
    import torch

    rng = np.random.default_rng(power)
    heads, dim, page, width, run = 1, 64, 64, 40, 512
    L = width * page
    dt = getattr(torch, dtype)
    lead = np.concatenate([512 * i + rng.choice(run, n, replace=False)
                           for i, n in enumerate(counts)])
    for sign in (1, -1):
        # the other tokens' scores are -7 2^power
        key = np.full((L, heads, dim), -448.0)
        key[lead] = sign * 64.0
        value = rng.standard_normal((L, heads, dim)) * 100
        value[lead] = np.where(lead % 2 == 0, 64.0, -8.0)[:, None, None]
        model = M.Cache(width, page, heads, dim)
        for n, x in (("k", key), ("v", value)):
            model.code[n] = M.encode(x).reshape(width, page, heads, dim).transpose(0, 2, 1, 3)
        model.exp["k"][:], model.exp["v"][:] = -6, -3
        cache = upload(S, model)
        scale = 2.0 ** (power - 6)  # 64 dims of q = 1 and |k| = 1
        values = model.values("v", np.arange(width), L)[0][:, 0]
        want = values[lead].mean(0)
        tol = torch.finfo(dt).eps / 2 * np.abs(want) + \
            np.abs(values[lead]).mean(0) * (2.0 ** -11 + (L / 32 + 64) * 2.0 ** -23)
        q = torch.ones((1, 1, 2, dim), dtype=dt, device="cuda")
        for B in (1, 800):  # split; as many requests as the card takes without
            table = i32(np.arange(width)[None].repeat(B, 0))
            out = cache.attend(q.expand(B, 1, 2, dim), table, i32([L] * B), scale=scale)
            got = out.double().cpu().numpy()
            assert (np.abs(got - want) <= tol).all(), (sign, B, got[0, 0, 0, 0], want[0])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_nan_key_among_growing_scores(S, dtype):
    """A NaN key in a tile that every row of its request sees, before and after tiles that move the
    maximum: that request is NaN, the other is not."""
    import torch

    rng = np.random.default_rng(23)
    heads, dim, page, width = 1, 128, 64, 6
    L = 300
    cache, model = filled(S, rng, 2 * width, page, heads, dim)
    base = np.sign(rng.standard_normal(dim))
    grow = np.linspace(0, 200, width * page)[:, None, None] * base
    for b in range(2):
        model.code["k"][b * width:(b + 1) * width] = M.encode(grow).reshape(
            width, page, heads, dim).transpose(0, 2, 1, 3)
    table = np.arange(2 * width).reshape(2, width)
    q = dev(np.tile(base, (2, 3, 4, 1))).to(getattr(torch, dtype))
    for tok in (0, 130, 250):
        keep = model.code["k"].copy()
        model.code["k"][table[0][tok // page], :, tok % page, 7] = 255
        out = upload(S, model).attend(q, i32(table), i32([L, L]))
        model.code["k"] = keep
        assert torch.isnan(out[0]).all()
        compare(out[1:], model, q[1:], table[1:], [L], None, dim ** -0.5, 0, 0)


def test_gradients_are_refused(S):
    """There is no backward: a tensor that asks for one is refused where it would be dropped
    without a word, and taken where gradients are off."""
    import torch

    cache = S.KVCache(1, 32, 1, 64)
    table, one = i32([[0]]), i32([1])
    x = torch.ones((1, 1, 1, 64), dtype=torch.float16, device="cuda")
    g = x.clone().requires_grad_()
    y = g * 2  # not a leaf
    for call in (lambda: cache.attend(g, table, one), lambda: cache.attend(y, table, one),
                 lambda: cache.write(g, x, table, i32([0])),
                 lambda: cache.write(x, y, table, i32([0])),
                 lambda: cache.read(table, i32([0]), None, 1, torch.float16, k=g, v=x)):
        with pytest.raises(RuntimeError, match="requires grad"):
            call()
    assert not cache.k.any().item() and not cache.v.any().item()
    with torch.no_grad():
        cache.write(g, y, table, i32([0]))
        assert torch.equal(cache.attend(g, table, one), 2 * x)
    assert torch.equal(cache.attend(g.detach(), table, one), 2 * x)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts(S, dim):
    """Prompts of a thousand tokens attend over themselves, from an empty cache and behind a
    prefix, with and without a window."""
    import torch

    rng = np.random.default_rng(dim)
    heads, group, page, width, T = 1, 2, 64, 20, 1030
    cache, model = filled(S, rng, 2 * width, page, heads, dim)
    table = rng.permutation(2 * width).reshape(2, width)
    q = dev(rng.standard_normal((2, T, heads * group, dim))).to(torch.bfloat16)
    for lens, qlens, window, sinks in (([1030, 1200], [1030, 1001], 0, 0),
                                       ([1030, 1200], [1030, 1001], 200, 4)):
        out = cache.attend(q, i32(table), i32(lens), i32(qlens), window=window, sinks=sinks)
        compare(out, model, q, table, lens, qlens, dim ** -0.5, window, sinks)


def test_short_requests_in_a_wide_table(S):
    """A table sized for the longest allowed context, mostly unmapped, with short requests."""
    import torch

    rng = np.random.default_rng(24)
    heads, group, dim, page, T = 2, 4, 128, 128, 5
    cache, model = filled(S, rng, 16, page, heads, dim)
    table = np.full((2, 1024), -1)
    table[:, :8] = rng.permutation(16).reshape(2, 8)
    q = dev(rng.standard_normal((2, T, heads * group, dim))).to(torch.float16)
    for lens in ([1000, 37], [129, 1024]):
        out = cache.attend(q, i32(table), i32(lens))
        compare(out, model, q, table, lens, None, dim ** -0.5, 0, 0)
