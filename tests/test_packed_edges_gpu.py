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


# ------------------------------------------------------------------ plans that only long inputs reach
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("lens,heads,dim", [([8192], 8, 128), ([5000, 3190], 8, 128),
                                            ([2049, 2047, 4100], 8, 64), ([4000, 3990], 4, 256)])
def test_prompts_cut_in_two(S, lens, heads, dim, dtype):
    """Row tiles that fill the card just once: those that see more than 32 token tiles come in two parts,
    the others in one.  Rows on both sides of every such border (2048 tokens at 64 and 128 dims, 1024 at
    256), of the tiles of rows and of the second part."""
    offsets = [0] + np.cumsum(lens).tolist()
    N = offsets[-1]
    size = ctypes.c_size_t()
    assert S.load().sfx_prompt_attention_workspace_bytes(len(lens), N, heads, heads, dim, 0, 0,
                                                         ctypes.byref(size)) == S.OK
    assert size.value == 2 * N * heads * (dim + 2) * 4   # two parts
    q, k, v = (rand(i, N, heads, dim, dtype=dtype) for i in range(3))
    out = S.attend_prompt(q, k, v, i32(offsets))
    rows = [0, 127, 128, 255, 256, 1023, 1024, 1025, 1151, 1152, 2047, 2048, 2049, 2303, 2304, 3071,
            3999, 4095, 4096, 4999, 8191]
    check_rows(out, q, k, v, offsets, rows)
    # a window moves the border: 3000 tokens are 47 tiles for every row that far in
    out = S.attend_prompt(q, k, v, i32(offsets), window=3000)
    check_rows(out, q, k, v, offsets, rows, window=3000)


def cached_rows(q, cache, table, length, n, lo, rows, window=0, sinks=0):
    """Definition in 64 bits over the values that the cache holds, of rows `rows` of the n newest tokens
    of a request (its first in row lo of q)."""
    import torch

    k, v = cache.read(table, i32([0]), i32([length]), length, dtype=torch.float32)
    mapped = ((table[0] >= 0) & (table[0] < cache.num_pages)).cpu()
    group = q.shape[1] // cache.kv_heads
    kk, vv = (t[0].double().cpu().repeat_interleave(group, 1) for t in (k, v))
    j = torch.arange(length)
    out, mag, dots = [], [], []
    for t in rows:
        p = length - n + t
        see = (j <= p) & mapped[j // cache.page_size]
        if window:
            see &= (j > p - window) | (j < sinks)
        x = q[lo + t].double().cpu()[None]
        s = (kk[see] * x).sum(2) * q.shape[2] ** -0.5
        w = (s - s.amax(0)).exp()
        w /= w.sum(0)
        out.append((w[:, :, None] * vv[see]).sum(0))
        mag.append((w[:, :, None] * vv[see].abs()).sum(0))
        dots.append((kk[see].abs() * x.abs()).sum(2).amax(0) * q.shape[2] ** -0.5)
    return torch.stack(out), torch.stack(mag), torch.stack(dots)[:, :, None], float(vv.abs().max())


def check_cached(got, ref, length, dim):
    """Tolerance: the result's rounding, eps / 2 of it; in units of sum p |v| each weight's to fp16,
    2^-11 (below 2^-22 of the largest to a multiple of 2^-33 of it), the scores' fp32 error and the
    sums' as for prompts."""
    import torch

    ref, mag, dots, most = ref
    eps = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu()
    rel = 2.0 ** -11 + 2 * (dim + 8) * 2.0 ** -24 * (dots + 1) + (length / 16 + 64) * 2.0 ** -23
    tol = eps * ref.abs() + mag * rel + length * 2.0 ** -33 * most
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= tol).all(), ((err > tol).nonzero()[:4].tolist(), float((err - tol).max()))


@pytest.mark.parametrize("dim,page,group", [(64, 32, 4), (128, 64, 4), (128, 96, 2), (256, 2048, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5000, 200)])
def test_chunks_over_many_pages(S, dim, page, group, window, sinks):
    """A chunk whose workgroups walk thousands of tokens in one part: page ids and scales are fetched 64
    blocks at a time, several times.  Pages without order, some unmapped."""
    heads, length, n = 8, 7300, 2400
    width = length // page + 2
    cache = S.KVCache(width, page, heads, dim)
    rng = np.random.default_rng(dim + page)
    table = i32(rng.permutation(width)[None])
    k, v = (rand(i, 1, length, heads, dim) for i in (1, 2))
    # tokens of all sizes: neighbouring blocks have other exponents
    size = (rand(3, 1, length // 32 + 1, heads, 1).float() * 2).exp2().repeat_interleave(32, 1)
    cache.write(k, (v.float() * size[:, :length]).half(), table, i32([0]))
    for j in ((1, 40, 70, 71, 150, 200) if width > 100 else (1,)):
        if j < width:
            table[0, j] = -1
    q = rand(4, n, heads * group, dim)
    out = cache.attend_packed(q, table, i32([length]), i32([0, n]), window=window, sinks=sinks)
    rows = [0, 1, 63, 64, 127, 128, 700, 1500, n - 1]
    ref = cached_rows(q, cache, table, length, n, 0, rows, window, sinks)
    check_cached(out[rows], ref, length, dim)


@pytest.mark.parametrize("heads,N", [(4, 9001), (9, 9000), (16, 9001), (40, 4096)])
def test_write_slots_of_large_batches(S, heads, N):
    """A wavefront looks at 8 to 32 tokens: stretches that begin at the last of them and end with the last
    slot read, single tokens, gaps; as the padded write does it."""
    import torch

    dim, page = 64, 64
    assert 4 < N * heads // 4096
    rng = np.random.default_rng(N + heads)
    # the first prompt's blocks all begin at rows 31, 63, ..: the last of a window of 32, or of 8
    lens, start = [1, 30, 2050], [70, 1, 0]
    while sum(lens) < N - 100:
        lens.append(min(N - 100 - sum(lens), int(rng.choice([1, 1, 17, 31, 33, 300, 1500]))))
        start.append(int(rng.integers(0, 100)))
    B, width = len(lens), 36
    table = rng.permutation(B * width).reshape(B, width)
    slots = np.full(N, -1, np.int64)
    off, at = [], 0
    for b, n in enumerate(lens):
        at += int(b > 2 and rng.random() < 0.2 and at + 1 + sum(lens[b:]) <= N)
        off.append(at)
        p = np.arange(start[b], start[b] + n)
        slots[at:at + n] = table[b, p // page] * page + p % page
        at += n
    a, b = S.KVCache(B * width, page, heads, dim), S.KVCache(B * width, page, heads, dim)
    for name in ("k", "v"):
        fill = torch.randint(0, 120, getattr(a, name).shape, dtype=torch.uint8, device="cuda")
        getattr(a, name).copy_(fill)
        getattr(b, name).copy_(fill)
        for c in (a, b):
            getattr(c, name + "_scale").fill_(2.0 ** -9)
    k, v = rand(1, N, heads, dim), rand(2, N, heads, dim)
    a.write_slots(k, v, torch.from_numpy(slots).cuda())
    for i, n in enumerate(lens):
        b.write(k[None, off[i]:off[i] + n], v[None, off[i]:off[i] + n], i32(table[i:i + 1]),
                i32(start[i:i + 1]))
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_a_cache_past_4_gib(S):
    """Pages whose codes lie past 2^32 bytes: written by slots, attended by short and long requests, as
    the same tokens in a small cache."""
    import torch

    heads, dim, page, group, pages = 8, 128, 64, 2, 70000
    far, near = S.KVCache(pages, page, heads, dim), S.KVCache(24, page, heads, dim)
    assert far.k.numel() > 2 ** 32
    last = np.arange(pages - 24, pages)
    order = np.random.default_rng(1).permutation(24).reshape(2, 12)
    N, lens, count = 700, [700, 300], [500, 200]
    k, v, q = (rand(i, N, h, dim) for i, h in enumerate((heads, heads, heads * group)))
    out = []
    for cache, ids in ((far, last), (near, np.arange(24))):
        table = i32(ids[order])
        pool = S.PagePool(cache.num_pages, page)
        for start, n in (([0, 0], [200, 100]), ([200, 100], count)):
            lay = pool.layout(table, i32(start), i32(n), N)
            cache.write_slots(k, v, lay.slots)
        assert lay.seq_lens.tolist() == lens
        out.append([cache.attend_packed(q, table, lay.seq_lens, lay.offsets),
                    cache.attend_packed(q[:4], table, lay.seq_lens, i32([0, 1, 4]), max_q=3)])
    for a, b in zip(*out):
        assert torch.equal(a, b) and a.abs().sum() > 0
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(far, name)[pages - 24:], getattr(near, name)), name
    assert not far.k[:1000].any() and not far.v[:1000].any()


def test_the_same_bits_every_time(S):
    """Calls again, on another stream and beside another call of the same shapes: the same results."""
    import torch

    heads, group, dim, page = 2, 4, 128, 64
    cache = cached(S, 3, 80, page, heads, dim, dtype="bfloat16")
    table = i32(np.random.default_rng(2).permutation(80).reshape(4, 20))
    offsets, lens = i32([0, 600, 617, 618, 700]), i32([1200, 900, 40, 82])
    q, k, v = (rand(i, 700, h, dim, dtype="bfloat16") for i, h in ((1, 8), (2, heads), (3, heads)))
    prompts = i32([0, 100, 650, 700])

    def both(stream=None):
        return (cache.attend_packed(q, table, lens, offsets, stream=stream),
                S.attend_prompt(q, k, v, prompts, stream=stream))

    want = both()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [both(st) for _ in range(5) for st in streams]
    torch.cuda.synchronize()
    for x in got + [both()]:
        assert all(torch.equal(a, b) for a, b in zip(x, want))


def test_pages_stay_within_their_arrays(S):
    """The list of free pages, the table and the counts lie between words that nobody may write; counts that
    cannot be are clamped."""
    import torch

    B, width, pages = 2, 4, 8
    whole = torch.full((400,), 7, dtype=torch.int32, device="cuda")
    at = dict(free=(64, pages), num_free=(128, 1), table=(150, B * width), held=(200, B),
              tokens=(250, B), missing=(300, B))
    a = {n: whole[i:i + size] for n, (i, size) in at.items()}
    a["free"].copy_(i32(np.arange(pages)))
    edge = torch.ones(400, dtype=torch.bool, device="cuda")
    for i, size in at.values():
        edge[i:i + size] = False
    pool = S.PagePool(pages, 64, buffers=(a["free"], a["num_free"]))
    table = a["table"].view(B, width)
    for num_free, held, tokens, missing in ((100, [-5, 99], [256, 0], [0, 0]),
                                            (2 ** 31 - 1, [99, 99], [0, 0], [0, 0]),
                                            (-2 ** 31, [0, 0], [64, 64], [1, 1]),
                                            (8, [-2 ** 31, 2 ** 31 - 1], [2 ** 31 - 1, -1],
                                             [2 ** 25, 0])):
        table.copy_(i32(np.arange(B * width).reshape(B, width)))
        a["num_free"].fill_(num_free)
        a["held"].copy_(i32(held))
        a["tokens"].copy_(i32(tokens))
        got = pool.reserve(table, a["held"], a["tokens"], missing=a["missing"])
        assert got.tolist() == missing
        assert whole[edge].eq(7).all()
        assert 0 <= int(a["num_free"]) <= pages
    for kw in (dict(tokens=a["held"]), dict(missing=a["held"]), dict(missing=a["tokens"])):
        args = dict(dict(held=a["held"], tokens=a["tokens"], missing=a["missing"]), **kw)
        with pytest.raises(ValueError, match="of their own"):
            pool.reserve(table, **args)


@pytest.mark.parametrize("group", [100, 192, 193, 300])
def test_many_query_heads_of_one(S, group):
    """More query heads of a cached one than the kernel of few rows takes: single tokens and short
    requests then are rows like any other."""
    dim, page, lens, n = 64, 32, [70, 1, 333], [1, 1, 5]
    cache = cached(S, group, 36, page, 1, dim)
    table = i32(np.random.default_rng(group).permutation(36).reshape(3, 12))
    offsets = [0, 1, 2, 7]
    q = rand(1, 9, group, dim)
    for max_q in (None, 5, 1):
        out = cache.attend_packed(q, table, i32(lens), i32(offsets), max_q=max_q)
        for b in range(3):
            live = min(n[b], max_q or 9)
            ref = cached_rows(q, cache, table[b:b + 1], lens[b], n[b], offsets[b], range(live))
            check_cached(out[offsets[b]:offsets[b] + live], ref, lens[b], dim)
            assert out[offsets[b] + live:offsets[b + 1]].eq(0).all()
        assert out[7:].eq(0).all()
    k, v = rand(2, 9, 1, dim), rand(3, 9, 1, dim)
    out = S.attend_prompt(q, k, v, i32(offsets))
    check_rows(out, q, k, v, offsets, range(5))


def test_seventy_thousand_requests(S):
    """Single tokens, requests without any and two longer ones, as the padded calls do them."""
    import torch

    B, dim, page = 70000, 64, 32
    rng = np.random.default_rng(7)
    n = rng.integers(0, 2, B)
    n[100], n[B - 1] = 9, 300
    offsets = np.concatenate([[0], np.cumsum(n)]) + 3
    N = int(offsets[-1]) + 4
    tokens = np.where(n > 0, n + rng.integers(0, 20, B), 0)
    pool = S.PagePool(B + 40, page)
    table, held = i32(np.full((B, 10), -1)), i32(np.zeros(B))
    assert not pool.reserve(table, held, i32(tokens)).any()
    assert held.tolist() == (-(-tokens // page)).tolist()
    lay = pool.layout(table, i32(tokens - n), i32(n), N)
    assert lay.offsets.tolist() == (offsets - 3).tolist() and lay.seq_lens.tolist() == tokens.tolist()
    cache = S.KVCache(B + 40, page, 1, dim)
    k, v = rand(1, 1, 32, 1, dim), rand(2, 1, 32, 1, dim)
    ids = torch.arange(B + 40, dtype=torch.int32, device="cuda")[:, None]
    cache.write(k.expand(B + 40, 32, 1, dim), v.expand(B + 40, 32, 1, dim), ids,
                torch.zeros_like(ids[:, 0]))
    q = rand(3, N, 2, dim)
    for max_q in (None, 300):
        out = cache.attend_packed(q, table, lay.seq_lens, lay.offsets, max_q=max_q)
        one = torch.from_numpy(np.flatnonzero(n == 1)).cuda()
        rows = lay.offsets[one].long()
        want = cache.attend(q[rows][:, None], table[one].contiguous(), lay.seq_lens[one])[:, 0]
        assert (out[rows].float() - want.float()).abs().max() <= 2.0 ** -9 * want.abs().max()
        for b in (100, B - 1):
            lo, hi = int(lay.offsets[b]), int(lay.offsets[b + 1])
            want = cache.attend(q[None, lo:hi], table[b:b + 1], lay.seq_lens[b:b + 1])[0]
            assert (out[lo:hi].float() - want.float()).abs().max() <= 2.0 ** -9 * want.abs().max()
        assert out[int(lay.offsets[-1]):].eq(0).all()
    # prompts of one token see themselves alone
    k, v = rand(4, N, 1, dim), rand(5, N, 1, dim)
    out = S.attend_prompt(q, k, v, lay.offsets)
    assert torch.equal(out[rows], v[rows].expand(-1, 2, -1))
