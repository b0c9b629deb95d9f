"""Packed batches at the edges of what the header allows: outputs that are left out, memory that is
shared, the largest values, plans that only long inputs reach."""
import ctypes

import numpy as np
import pytest

from tests import packed_model as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import suffix_match_drafter_amd as sfx

    sfx.load()
    return sfx


def i32(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


# ------------------------------------------------------------------ the layout
@pytest.mark.parametrize("wanted", ["seq_lens", "request", "position", "slots"])
def test_layout_of_one_output(S, wanted):
    """Each of the last four outputs by itself; the page table is given for slots only."""
    import torch

    start, count, N, page, pages = [60, 0, 5], [10, 0, 70], 90, 64, 6
    table = np.array([[3, 1], [2, 0], [5, 4]], np.int32)
    want = dict(zip(("offsets", "seq_lens", "request", "position", "slots"),
                    M.layout(table, start, count, N, page, pages)))
    out = torch.full((len(want[wanted]),), 77, device="cuda",
                     dtype=torch.int64 if wanted == "slots" else torch.int32)
    offsets = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    t, s, c = i32(table), i32(start), i32(count)
    at = [ctypes.c_void_p(out.data_ptr()) if name == wanted else None
          for name in ("seq_lens", "request", "position", "slots")]
    rc = S.load().sfx_step_layout(3, N, 2, page, pages, t.data_ptr() if wanted == "slots" else None,
                                  s.data_ptr(), c.data_ptr(), offsets.data_ptr(), *at, None)
    assert rc == S.OK
    torch.cuda.synchronize()
    assert offsets.tolist() == want["offsets"].tolist()
    assert out.tolist() == want[wanted].tolist()


# ------------------------------------------------------------------ the pages
@pytest.mark.parametrize("B", [5, 5000])
def test_missing_in_the_place_of_tokens(S, B):
    """The C call may leave what is missing where the lengths stood."""
    import torch

    rng = np.random.default_rng(B)
    page, width, pages = 16, 3, B
    tokens = rng.integers(0, width * page + 20, B)
    table, held = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    free = rng.permutation(pages).astype(np.int32)
    want = M.reserve(table, held, free, pages, tokens, page, pages)
    t, h, f, n, k = i32(table), i32(held), i32(free), i32([pages]), i32(tokens)
    size = ctypes.c_size_t()
    assert S.load().sfx_pages_reserve_workspace_bytes(B, width, ctypes.byref(size)) == S.OK
    ws = torch.empty(max(size.value, 16), dtype=torch.uint8, device="cuda")
    rc = S.load().sfx_pages_reserve(B, width, page, pages, k.data_ptr(), t.data_ptr(), h.data_ptr(),
                                    f.data_ptr(), n.data_ptr(), k.data_ptr(), ws.data_ptr(),
                                    size.value, None)
    assert rc == S.OK
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), want[0]) and h.tolist() == want[1].tolist()
    assert int(n) == want[3] and f[:want[3]].tolist() == want[2][:want[3]].tolist()
    assert k.tolist() == want[4].tolist()


def test_held_and_tokens_of_one_array(S):
    """Tensors that overlap without being the same are refused as well."""
    x = i32(np.zeros(9))
    table = i32(np.full((8, 2), -1))
    pool = S.PagePool(4, 64)
    for kw in (dict(held=x[:8], tokens=x[1:]), dict(held=x[:8], tokens=i32(np.ones(8)),
                                                  missing=x[1:])):
        with pytest.raises(S.SfxError, match="share memory"):
            pool.reserve(table, **kw)
    one = i32([0])
    pool = S.PagePool(1, 64, buffers=(one, one))
    with pytest.raises(S.SfxError, match="share memory"):
        pool.reserve(i32([[-1]]), i32([0]), i32([1]))
    assert one.tolist() == [0] and x.tolist() == [0] * 9


@pytest.mark.parametrize("B", [3, 50000])
def test_more_pages_than_there_are(S, B):
    """Counts that contradict each other (every page free, some held all the same): the list takes what
    it has room for, and nothing passes its end, nor 2^31 where it is that long."""
    import torch

    tokens, held = i32(np.zeros(B)), i32(np.ones(B))
    tokens[0] = 64 * 2
    table = i32(np.arange(3 * B).reshape(B, 3))
    for pages in (2 ** 31 - 1, 40):
        whole = torch.empty(pages + 64, dtype=torch.int32, device="cuda")
        whole[pages:] = 77
        whole[:64] = 77
        pool = S.PagePool(pages, 64, buffers=(whole[:pages], i32([2 ** 31 - 1])))
        t, h = table.clone(), held.clone()
        assert pool.reserve(t, h, tokens).tolist() == [0] * B
        assert h.tolist() == [2] + [0] * (B - 1)
        # the first request's second page is the first one released, the others have no room left
        assert t[0].tolist() == [0, 3, 2] and t[1:, 0].eq(-1).all() and t[1:, 1:].equal(table[1:, 1:])
        assert int(pool.num_free) == pages
        assert whole[pages:].eq(77).all()
        assert whole[:min(64, pages)].eq(77).all()
        del pool, whole


# ------------------------------------------------------------------ attention
def rand(seed, *shape, dtype="float16"):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(getattr(torch, dtype))


def cached(S, seed, pages, page, heads, dim, dtype="float16"):
    """A cache with every page written, from tokens of one request."""
    cache = S.KVCache(pages, page, heads, dim)
    k, v = (rand(seed + i, 1, pages * page, heads, dim, dtype=dtype) for i in (0, 1))
    cache.write(k, v, i32(np.arange(pages)[None]), i32([0]))
    return cache


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_results_in_the_queries_place(S, dim):
    """out = q: short requests, chunks, rows of no request, parts that are joined."""
    import torch

    for offsets, group in (([3, 4, 21, 321, 330], 4), ([0, 1, 2], 1), ([0, 30, 60, 90], 2),
                           ([0, 700, 701], 1)):
        N, B = offsets[-1] + 2, len(offsets) - 1
        cache = cached(S, dim, 16 * B, 64, 1, dim)
        table = i32(np.random.default_rng(dim).permutation(16 * B).reshape(B, 16))
        lens, off = i32(np.maximum(np.diff(offsets), 1000 - 70 * np.arange(B))), i32(offsets)
        q, k, v = rand(5, N, group, dim), rand(6, N, 1, dim), rand(7, N, 1, dim)
        for max_q in (None, int(np.diff(offsets).max())):
            want = cache.attend_packed(q, table, lens, off, max_q=max_q)
            x = q.clone()
            assert cache.attend_packed(x, table, lens, off, max_q=max_q, out=x) is x
            assert torch.equal(x, want)
        want = S.attend_prompt(q, k, v, off)
        x = q.clone()
        assert S.attend_prompt(x, k, v, off, out=x) is x
        assert torch.equal(x, want)


def test_results_over_keys_or_values(S):
    """Refused: other workgroups still read them."""
    q, k, v = (rand(i, 40, 2, 64) for i in range(3))
    for bad in (k, v):
        was = bad.clone()
        with pytest.raises(S.SfxError, match="share memory"):
            S.attend_prompt(q, k, v, i32([0, 40]), out=bad)
        assert bad.equal(was)
    wide = rand(9, 41, 2, 64)
    with pytest.raises(S.SfxError, match="share memory"):
        S.attend_prompt(wide[1:], k, v, i32([0, 40]), out=wide[:40])


def prompt_rows(q, k, v, lo, rows, scale, window=0):
    """Definition in 64 bits of rows `rows` of a prompt that begins at row lo, with sum p |v| and the
    largest |q||k| scale."""
    import torch

    group = q.shape[1] // k.shape[1]
    kk = k.double().cpu().repeat_interleave(group, 1)
    vv = v.double().cpu().repeat_interleave(group, 1)
    out, mag, dots = [], [], []
    for t in rows:
        first = max(lo, t - window + 1) if window else lo
        x = q[t].double().cpu()[None]
        s = (kk[first:t + 1] * x).sum(2) * scale
        w = (s - s.amax(0)).exp()
        w /= w.sum(0)
        out.append((w[:, :, None] * vv[first:t + 1]).sum(0))
        mag.append((w[:, :, None] * vv[first:t + 1].abs()).sum(0))
        dots.append((kk[first:t + 1].abs() * x.abs()).sum(2).amax(0) * scale)
    return torch.stack(out), torch.stack(mag), torch.stack(dots)[:, :, None]


def check_rows(out, q, k, v, offsets, rows, scale=None, window=0, least=0.0):
    """`rows` of each request of a prompt call.  Tolerance: the result's rounding, eps / 2 of it; in units
    of sum p |v| each weight's rounding to the values' type, eps / 2 (fp16: to a multiple of 2^-33 of the
    largest below 2^-22 of it, once a token), the scores' fp32 error, (dim + 8) 2^-24 of |q||k| scale
    and their own size, twice, and the sums', 2^-23 per 16 tokens and 64 more; `least` absolutely."""
    import torch

    eps = torch.finfo(out.dtype).eps / 2
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    for b in range(len(offsets) - 1):
        lo, n = offsets[b], offsets[b + 1] - offsets[b]
        mine = [lo + r for r in rows if r < n]
        if not mine:
            continue
        ref, mag, dots = prompt_rows(q, k, v, lo, mine, scale, window)
        got = out[mine].double().cpu()
        assert torch.isfinite(got).all(), b
        rel = eps + 2 * (dim + 8) * 2.0 ** -24 * (dots + 1) + (n / 16 + 64) * 2.0 ** -23
        tol = eps * ref.abs() + mag * rel + least
        if out.dtype is torch.float16:
            tol = tol + n * 2.0 ** -33 * float(v[lo:lo + n].abs().max())
        err = (got - ref).abs()
        assert (err <= tol).all(), (b, (err > tol).nonzero()[:4].tolist(), float((err - tol).max()))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1, 2, 40], [1000, 3], [9000]])
def test_the_whole_range_of_bf16_values(S, lens, dim):
    """Values up to the type's largest, and down to small ones: weights of any size keep sums in range."""
    import torch

    offsets = [0] + np.cumsum(lens).tolist()
    N = offsets[-1]
    q, k = (rand(i, N, h, dim, dtype="bfloat16") for i, h in ((1, 2), (2, 1)))
    v = rand(3, N, 1, dim, dtype="bfloat16").clamp(-4, 4)
    rows = [0, 1, 2, 31, 32, 39, 63, 64, 700, 999, 4095, 8191, 8999]
    big = v * 2.0 ** 125    # up to 2^127
    check_rows(S.attend_prompt(q, k, big, i32(offsets)), q, k, big, offsets, rows)
    same = v.new_full(v.shape, 3e38)
    out = S.attend_prompt(q, k, same, i32(offsets))
    check_rows(out, q, k, same, offsets, rows)
    # even weights are powers of two: the largest value comes out as it is
    most = v.new_full(v.shape, torch.finfo(v.dtype).max)
    assert S.attend_prompt(q * 0, k, most, i32(offsets)).eq(most[0, 0, 0]).all()
    # scores that rise by less than it takes to move the maximum, then by more
    q0, k0 = torch.zeros_like(q), torch.zeros_like(k)
    q0[:, :, 0] = 1
    for step in (0.004, 0.05, 0.5):
        k0[:, 0, 0] = (torch.arange(N, device="cuda") * step).to(torch.bfloat16)
        out = S.attend_prompt(q0, k0, big, i32(offsets), scale=1.0)
        check_rows(out, q0, k0, big, offsets, rows, scale=1.0)
    # small values: as long as products with the weights are normal numbers nothing is lost
    small = v * 2.0 ** -90
    check_rows(S.attend_prompt(q, k, small, i32(offsets)), q, k, small, offsets, rows)
