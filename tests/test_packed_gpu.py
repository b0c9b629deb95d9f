"""Packed batches over the 8-bit cache: the write by slots against the model (codes and scales exactly)
and the attention against the definition in 64 bits, over the values that the cache holds.

Tolerance of one output o = sum p v, from the kernel's roundings:
  the result's own rounding, eps/2 of |o|;
  each weight p rounded to fp16, 2^-11 of it, and below 2^-22 of the largest weight to a multiple
  of 2^-33 of it at worst, once per token;
  a score's fp32 error: (dim + 8) 2^-24 of sum |q||k| scale plus its own size, twice (numerator
  and denominator), as a relative error of the weights;
  fp32 sums: one rounding of 2^-23 per 16 tokens, 64 more in and after the matrix product;
all but the first in units of A = sum p |v|."""
import numpy as np
import pytest

from tests import kv_model as K
from tests import packed_model as M

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
    model = K.Cache(pages, page, heads, dim)
    for n in "kv":
        model.code[n] = K.encode(rng.standard_normal(model.shape) * 60)
        model.exp[n] = rng.integers(-8 - spread, -7 + spread, size=model.exp[n].shape)
    return upload(S, model), model


def upload(S, model):
    P, H, page, d = model.shape
    bufs = [None] * 4
    for i, n in enumerate("kv"):
        c, s = model.pack(n)
        bufs[i], bufs[2 + i] = dev(c), dev(s)
    return S.KVCache(P, page, H, d, buffers=tuple(bufs))


def same(cache, model):
    """Scales equal; codes as values: a NaN has no sign in this format, nor has a zero."""
    for n in "kv":
        c, s = model.pack(n)
        a, b = K.VALUES[getattr(cache, n).cpu().numpy()], K.VALUES[c]
        bad = ~((a == b) | (np.isnan(a) & np.isnan(b)))
        assert not bad.any(), (n, np.argwhere(bad)[:5], a[bad][:5], b[bad][:5])
        assert (getattr(cache, n + "_scale").cpu().numpy() == s).all(), n


def compare(got, model, q, table, lens, offsets, max_q=None, window=0, sinks=0, scale=None):
    import torch

    eps = torch.finfo(got.dtype).eps / 2
    dim = model.shape[3]
    scale = dim ** -0.5 if scale is None else scale
    got, q = got.double().cpu().numpy(), q.double().cpu().numpy()
    covered = np.zeros(len(got), bool)
    for b in range(len(lens)):
        lo, hi = offsets[b], offsets[b + 1]
        if hi <= lo:
            continue
        ref, mag, dots = K.attention(model, q[lo:hi], table[b], lens[b], hi - lo, scale, window,
                                     sinks)
        if max_q is not None:
            ref[max_q:], mag[max_q:] = 0, 0
        L = max(lens[b], 1)
        rel = 2.0 ** -11 + 2 * (dim + 8) * 2.0 ** -24 * (dots + 1)[:, :, None] + \
            (L / 16 + 64) * 2.0 ** -23
        tol = eps * np.abs(ref) + mag * rel + (mag > 0) * L * 2.0 ** -33 * max(
            mag.max(), np.abs(K.VALUES[:127]).max() * 2.0 ** int(model.exp["v"].max()))
        assert np.isfinite(got[lo:hi]).all(), b
        err = np.abs(got[lo:hi] - ref)
        assert (err <= tol).all(), (b, np.argwhere(err > tol)[:4], err.max())
        covered[lo:hi] = True
    assert (got[~covered] == 0).all()


# ------------------------------------------------------------------ write by slots
def slots_of(table, start, lens, page):
    return np.concatenate([[table[b, p // page] * page + p % page for p in range(a, a + n)]
                           for b, (a, n) in enumerate(zip(start, lens))] + [[]]).astype(np.int64)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 32), (2, 128, 96), (3, 256, 64)])
@pytest.mark.parametrize("lens", [[1], [17, 1, 0, 33], [5, 64, 31, 32, 100], [1] * 70])
def test_write_slots(S, heads, dim, page, lens, dtype):
    import torch

    rng = np.random.default_rng(sum(lens) + dim)
    B, n = len(lens), sum(lens)
    width = 400 // page + 1
    cache, model = filled(S, rng, B * width, page, heads, dim)
    table = rng.permutation(B * width).reshape(B, width)
    start = [int(rng.choice([0, 1, 31, 32, 63, 100, 200])) for _ in lens]
    slots = slots_of(table, start, lens, page)
    x = [dev(rng.standard_normal((n, heads, dim)) * np.exp(rng.normal(size=(n, heads, 1)) * 2))
         .to(getattr(torch, dtype)) for _ in "kv"]
    cache.write_slots(*x, dev(slots))
    off = np.concatenate([[0], np.cumsum(lens)])
    for name, t in zip("kv", x):
        t = t.double().cpu().numpy()
        for b in range(B):
            model.write(name, t[off[b]:off[b + 1]], table[b], start[b], lens[b])
    same(cache, model)


@pytest.mark.parametrize("N", [9000, 4097])
def test_write_slots_many(S, N):
    """Prompts among single tokens, in a shuffled order of requests, as the padded write does it; with
    rows that go nowhere between and behind."""
    import torch

    rng = np.random.default_rng(N)
    heads, dim, page = 2, 64, 64
    lens, left = [], N - 300
    while left > 0:
        lens.append(min(left, int(rng.choice([1, 1, 1, 17, 300, 2000]))))
        left -= lens[-1]
    B = len(lens)
    width = 40
    start = [int(rng.integers(0, 100)) for _ in lens]
    table = rng.permutation(B * width).reshape(B, width)
    a, model = filled(S, rng, B * width, page, heads, dim)
    b = upload(S, model)
    k, v = (torch.randn((N, heads, dim), device="cuda").bfloat16() for _ in "kv")
    slots = np.full(N, -1, np.int64)
    off, at = [], 0
    gaps = rng.permutation([1] * 200 + [0] * B)
    for i, n in enumerate(lens):
        at += int(gaps[i])
        off.append(at)
        slots[at:at + n] = slots_of(table[i:i + 1], start[i:i + 1], [n], page)
        at += n
    free = np.flatnonzero(slots < 0)
    slots[free] = rng.choice([-1, -2 ** 62, B * width * page, 2 ** 40], size=len(free))
    a.write_slots(k, v, dev(slots))
    T = max(lens)
    rows = torch.tensor([[o + min(t, n - 1) for t in range(T)] for o, n in zip(off, lens)],
                        device="cuda")
    b.write(k[rows], v[rows], i32(table), i32(start), i32(lens))
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_write_slots_special(S):
    """Infinities saturate, NaN stays, zero blocks, strided inputs, nothing to write."""
    import torch

    rng = np.random.default_rng(1)
    cache, model = filled(S, rng, 4, 32, 2, 64)
    x = rng.standard_normal((40, 2, 64))
    x[3, 0, 5], x[4, 1, 7], x[38, 0, 0] = np.inf, np.nan, -np.inf
    x[20:30] = 0
    wide = torch.zeros((40, 5, 67), dtype=torch.float16, device="cuda")
    wide[:, 1:3, 2:66] = dev(x).half()
    t = wide[:, 1:3, 2:66]
    slots = np.concatenate([np.arange(32, 52), np.arange(100, 120)])
    cache.write_slots(t, t, dev(slots))
    h = t.double().cpu().numpy()
    for n in "kv":
        model.write(n, h[:20], [1], 0, 20)
        model.write(n, h[20:], [3], 4, 20)
    same(cache, model)
    cache.write_slots(t[:0], t[:0], dev(slots[:0]))
    S.KVCache(0, 32, 2, 64).write_slots(t, t, dev(slots))
    same(cache, model)


# ------------------------------------------------------------------ attention
CASES = [
    # heads, group, dim, page, lens, rows, window, sinks
    (1, 1, 64, 32, [1], [1], 0, 0),
    (2, 4, 128, 64, [33, 1000, 31], [1, 1, 1], 0, 0),
    (2, 3, 64, 96, [5, 3], [5, 5], 0, 0),                # a row before the first token
    (1, 8, 128, 32, [9, 64, 200], [0, 9, 4], 0, 0),
    (2, 8, 128, 64, [17, 777, 40], [17, 16, 1], 0, 0),
    (1, 5, 256, 128, [500, 3], [33, 3], 0, 0),
    (2, 16, 256, 64, [3, 260], [2, 3], 0, 0),
    (1, 1, 64, 32, [300], [270], 0, 0),
    (1, 4, 128, 64, [600, 20, 400, 77], [200, 20, 17, 1], 0, 0),   # a chunk, a prompt, a draft
    (2, 2, 64, 32, [700, 90], [130, 3], 1, 0),                       # sees itself alone
    (1, 2, 128, 64, [700, 90], [130, 70], 100, 0),
    (1, 2, 128, 64, [700, 90], [4, 80], 33, 4),
    (1, 4, 64, 32, [900, 40], [100, 17], 64, 100),
    (2, 2, 64, 32, [640], [2], 5, 1000),
    (1, 2, 256, 32, [300, 1], [140, 1], 70, 3),
    (8, 1, 128, 2048, [4000, 10], [1, 2], 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_model(S, case, dtype):
    import torch

    heads, group, dim, page, lens, rows, window, sinks = case
    rng = np.random.default_rng(sum(lens) * 10 + dim)
    B = len(lens)
    width = max(lens) // page + 2
    cache, model = filled(S, rng, B * width, page, heads, dim)
    table = rng.permutation(B * width).reshape(B, width)
    offsets = np.concatenate([[0], np.cumsum(rows)])
    q = dev(rng.standard_normal((offsets[-1], heads * group, dim))).to(getattr(torch, dtype))
    args = (q, i32(table), i32(lens), i32(offsets))
    out = cache.attend_packed(*args, window=window, sinks=sinks)
    compare(out, model, q, table, lens, offsets, window=window, sinks=sinks)
    tight = cache.attend_packed(*args, max_q=max(rows), window=window, sinks=sinks)
    compare(tight, model, q, table, lens, offsets, window=window, sinks=sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_q", [0, 1, 5, 40, 129])
def test_rows_past_max_q(S, dim, max_q):
    """Rows of a request from max_q on, of no request and before the first one are zero; the others
    keep their positions."""
    import torch

    rng = np.random.default_rng(dim + max_q)
    page, heads, group = 64, 2, 4
    lens, rows = [400, 40, 0, 300], [150, 40, 3, 1]
    cache, model = filled(S, rng, 4 * 8, page, heads, dim)
    table = rng.permutation(32).reshape(4, 8)
    offsets = 30 + np.concatenate([[0], np.cumsum(rows)])
    q = dev(rng.standard_normal((260, heads * group, dim))).half()
    q[:30], q[offsets[-1]:] = float("nan"), float("nan")
    out = cache.attend_packed(q, i32(table), i32(lens), i32(offsets), max_q=max_q)
    compare(out, model, q, table, lens, offsets, max_q=max_q)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("rows", [1, 17, 300])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_and_split(S, dim, rows):
    """Long requests beside short ones, one head: parts over the tokens, some of them empty."""
    rng = np.random.default_rng(dim + rows)
    page, lens = 64, [3000, 5, 700, 64]
    n = [rows, 5, min(rows, 2), 1]
    cache, model = filled(S, rng, 4 * 50, page, 1, dim)
    table = rng.permutation(200).reshape(4, 50)
    offsets = np.concatenate([[0], np.cumsum(n)])
    q = dev(rng.standard_normal((offsets[-1], 2, dim))).half()
    for window, sinks in ((0, 0), (1500, 40)):
        for max_q in (None, max(n)):
            out = cache.attend_packed(q, i32(table), i32(lens), i32(offsets), max_q=max_q,
                                      window=window, sinks=sinks)
            compare(out, model, q, table, lens, offsets, window=window, sinks=sinks)


@pytest.mark.parametrize("B", [62, 63, 200])
def test_many_requests(S, B):
    """Single tokens and drafts around two chunks, some requests without rows."""
    rng = np.random.default_rng(B)
    page, heads, group, dim = 32, 2, 2, 64
    rows = rng.integers(0, 4, B)
    rows[3], rows[B - 2] = 210, 150
    lens = np.maximum(rows, rng.integers(1, 300, B))
    width = 300 // page + 1
    cache, model = filled(S, rng, B * width, page, heads, dim)
    table = rng.permutation(B * width).reshape(B, width)
    offsets = 2 + np.concatenate([[0], np.cumsum(rows)])
    q = dev(rng.standard_normal((int(offsets[-1]) + 3, heads * group, dim))).half()
    out = cache.attend_packed(q, i32(table), i32(lens), i32(offsets))
    compare(out, model, q, table, lens.tolist(), offsets)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("rows", [1, 20, 200])
def test_exponents_far_apart(S, rows, dtype):
    """Block exponents over their whole range: every value counts with its own power of two."""
    import torch

    rng = np.random.default_rng(rows)
    page, dim = 32, 64
    model = K.Cache(16, page, 1, dim)
    for n in "kv":
        model.code[n] = K.encode(rng.standard_normal(model.shape) * 60)
    # keys small enough for finite scores, values from the least to the largest exponent
    model.exp["k"] = rng.integers(-32, -7, size=model.exp["k"].shape)
    model.exp["v"] = rng.integers(-32, 32 if dtype == "bfloat16" else 5,
                                  size=model.exp["v"].shape)
    cache = upload(S, model)
    table, lens = np.arange(16)[None], [500]
    q = dev(rng.standard_normal((rows, 1, dim))).to(getattr(torch, dtype))
    out = cache.attend_packed(q, i32(table), i32(lens), i32([0, rows]))
    compare(out, model, q, table, lens, [0, rows])


@pytest.mark.parametrize("rows", [3, 150])
def test_unmapped_pages_and_nan(S, rows):
    """Unmapped pages are not seen, a request of none is zero; NaN values behind a row's position, past
    its window or past the request do not reach it."""
    import torch

    rng = np.random.default_rng(rows)
    page, dim, heads, group = 64, 128, 2, 2
    cache, model = filled(S, rng, 24, page, heads, dim)
    table = rng.permutation(24).reshape(3, 8)
    table[0, 2], table[0, 4], table[1] = -1, 99, -1
    lens = [450, 300, 250]
    offsets = [0, rows, 2 * rows, 3 * rows]
    q = dev(rng.standard_normal((3 * rows, heads * group, dim))).bfloat16()
    args = (q, i32(table), i32(lens), i32(offsets))
    out = cache.attend_packed(*args)
    compare(out, model, q, table, lens, offsets)
    assert out[rows:2 * rows].eq(0).all()
    # NaN codes in the tokens behind the request's last, and in one before it
    for p in range(250, 512):
        model.code["v"][table[2, p // page], :, p % page] = 127
        model.code["k"][table[2, p // page], :, p % page] = 127
    bad = 249 - rows // 2
    model.code["v"][table[2, bad // page], 0, bad % page, 9] = 255
    cache2 = upload(S, model)
    again = cache2.attend_packed(*args)
    assert torch.equal(again[:2 * rows], out[:2 * rows])
    first = 2 * rows + bad - (250 - rows)   # the first row that sees it
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[first:, :group, 9] = True
    assert again[hit].isnan().all() and torch.equal(again[~hit], out[~hit])


@pytest.mark.parametrize("rows", [1, 140])
@pytest.mark.parametrize("nan_page,gone", [(4, 5), (5, 4)])
def test_nan_beside_an_unmapped_page(S, rows, nan_page, gone):
    """A NaN value that every row sees, next to a page that is not mapped and holds NaN as well: the
    first reaches them all, the second nobody."""
    rng = np.random.default_rng(rows)
    plain, model = filled(S, rng, 20, 32, 1, 64)
    table = np.arange(20)[None].copy()
    table[0, gone] = -1
    q = dev(rng.standard_normal((rows, 1, 64))).half()
    args = (q, i32(table), i32([600]), i32([0, rows]))
    want = plain.attend_packed(*args)
    model.code["v"][[nan_page, gone], 0, 3, 7] = 127
    out = upload(S, model).attend_packed(*args)
    assert out[:, :, 7].isnan().all()
    assert out[:, :, :7].equal(want[:, :, :7]) and out[:, :, 8:].equal(want[:, :, 8:])


def test_as_the_padded_call(S):
    """Requests of one length: the padded attention's results, within both roundings."""
    import torch

    rng = np.random.default_rng(2)
    B, T, heads, group, dim, page = 5, 17, 2, 4, 128, 64
    cache, model = filled(S, rng, B * 12, page, heads, dim)
    table = i32(rng.permutation(B * 12).reshape(B, 12))
    lens = i32([700, 17, 300, 64, 500])
    q = dev(rng.standard_normal((B, T, heads * group, dim))).half()
    a = cache.attend(q, table, lens).flatten(0, 1)
    b = cache.attend_packed(q.flatten(0, 1), table, lens, i32(np.arange(B + 1) * T), max_q=T)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -9 * a.float().abs().max()


def test_strides_streams_and_graph(S):
    """A slice of a fused projection, another stream, a capture replayed with other lengths."""
    import torch

    rng = np.random.default_rng(3)
    heads, group, dim, page = 2, 4, 128, 64
    cache, _ = filled(S, rng, 40, page, heads, dim)
    table = i32(rng.permutation(40).reshape(4, 10))
    lens, offsets = i32([600, 100, 5, 300]), i32([0, 200, 217, 218, 230])
    wide = torch.randn((230, heads * (group + 2) * dim), device="cuda").half()
    q = wide[:, :heads * group * dim].unflatten(1, (heads * group, dim))
    assert not q.is_contiguous()
    want = cache.attend_packed(q.contiguous(), table, lens, offsets)
    assert torch.equal(cache.attend_packed(q, table, lens, offsets), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = cache.attend_packed(q, table, lens, offsets, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend_packed(q, table, lens, offsets, out=out)
    for i, (n, off) in enumerate((([600, 100, 5, 300], [0, 200, 217, 218, 230]),
                                  ([230, 0, 1, 9], [0, 230, 230, 230, 230]),
                                  ([630, 630, 630, 630], [3, 4, 5, 6, 100]))):
        lens.copy_(i32(n))
        offsets.copy_(i32(off))
        wide.copy_(torch.randn_like(wide))
        out.fill_(7)
        g.replay()
        got = out.clone()
        assert torch.equal(got, cache.attend_packed(q, table, lens, offsets)), i
        torch.cuda.synchronize()


# ------------------------------------------------------------------ the calls together
def test_steps_of_continuous_batching(S):
    """Requests come, grow by prompt chunks, drafts and single tokens, and end; every step runs reserve,
    layout, write_slots and attend_packed.  Each request's results are those of the model over a cache
    that it has for itself, whatever pages it was given."""
    import torch

    rng = np.random.default_rng(11)
    B, heads, group, dim, page, pages, N = 6, 1, 2, 64, 32, 20, 220
    cache, pool = S.KVCache(pages, page, heads, dim), S.PagePool(pages, page)
    table, held = i32(np.full((B, 16), -1)), i32(np.zeros(B))
    mine = [K.Cache(16, page, heads, dim) for _ in range(B)]
    seq = np.zeros(B, int)
    waited = 0
    for step in range(14):
        ends = rng.random(B) < 0.15
        seq[ends] = 0
        count = np.array([int(rng.choice([1, 1, 5, 17, 90])) if s else int(rng.integers(1, 100))
                          for s in seq])
        count = np.where(seq + count > 16 * page, 0, count)
        while count.sum() > N:
            count[rng.integers(B)] = 0
        missing = pool.reserve(table, held, i32(seq + count))
        count = np.where(missing.cpu().numpy() > 0, 0, count)   # those wait for a step
        waited += int((missing > 0).sum())
        lay = pool.layout(table, i32(seq), i32(count), N)
        k, v = (torch.randn((N, heads, dim), device="cuda").half() for _ in "kv")
        q = torch.randn((N, heads * group, dim), device="cuda").half()
        cache.write_slots(k, v, lay.slots)
        out = cache.attend_packed(q, table, lay.seq_lens, lay.offsets)
        off = lay.offsets.tolist()
        for b in range(B):
            for name, t in zip("kv", (k, v)):
                mine[b].write(name, t[off[b]:off[b + 1]].double().cpu().numpy(),
                              list(range(16)), int(seq[b]), int(count[b]))
        assert lay.seq_lens.tolist() == (seq + count).tolist()
        assert out[off[-1]:].eq(0).all()
        for b in range(B):
            lo, hi = off[b], off[b + 1]
            if hi > lo:
                compare(out[lo:hi], mine[b], q[lo:hi], [list(range(16))],
                        [int(seq[b] + count[b])], [0, hi - lo])
        # some of the drafted tokens are rejected: their places are written again
        keep = np.where(count > 1, np.maximum(1, count - rng.integers(0, 3, B)), count)
        seq = seq + keep
    assert waited > 0
    pool.reserve(table, held, i32(np.zeros(B)))
    assert sorted(pool.free.tolist()) == list(range(pages)) and int(pool.num_free) == pages


def test_a_prompt_both_ways(S):
    """attend_prompt over a prompt's own values and attend_packed over its cached ones: equal where the
    cache holds the values exactly."""
    import torch

    rng = np.random.default_rng(12)
    heads, group, dim, page, n = 2, 2, 128, 64, 333
    # whole numbers up to 8 are e4m3's
    k, v = (dev(rng.integers(-8, 9, (n, heads, dim))).half() for _ in "kv")
    q = dev(rng.standard_normal((n, heads * group, dim)) * 0.3).half()
    cache, pool = S.KVCache(8, page, heads, dim), S.PagePool(8, page)
    table, held = i32(np.full((2, 6), -1)), i32([0, 0])
    assert pool.reserve(table, held, i32([200, 133])).tolist() == [0, 0]
    lay = pool.layout(table, i32([0, 0]), i32([200, 133]), n)
    cache.write_slots(k, v, lay.slots)
    a = S.attend_prompt(q, k, v, lay.offsets)
    b = cache.attend_packed(q, table, lay.seq_lens, lay.offsets)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -9 * a.float().abs().max()


def test_captured_step(S):
    """The whole step in one graph, replayed with other lengths, against eager calls on a second set of
    buffers."""
    import torch

    rng = np.random.default_rng(13)
    B, heads, group, dim, page, pages, N = 4, 1, 4, 128, 64, 40, 150
    k, v = (torch.randn((N, heads, dim), device="cuda").half() for _ in "kv")
    q = torch.randn((N, heads * group, dim), device="cuda").half()
    start, count, tokens = (i32(np.zeros(B)) for _ in range(3))

    class Side:
        def __init__(self):
            self.cache, self.pool = S.KVCache(pages, page, heads, dim), S.PagePool(pages, page)
            self.table, self.held = i32(np.full((B, 10), -1)), i32(np.zeros(B))

        def step(self):
            self.missing = self.pool.reserve(self.table, self.held, tokens)
            self.lay = self.pool.layout(self.table, start, count, N)
            self.cache.write_slots(k, v, self.lay.slots)
            self.out = self.cache.attend_packed(q, self.table, self.lay.seq_lens,
                                                self.lay.offsets)

    a, b = Side(), Side()
    Side().step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step()
    seq = np.zeros(B, int)
    for i in range(5):
        n = rng.integers(0, 38, B)
        start.copy_(i32(seq))
        count.copy_(i32(n))
        tokens.copy_(i32(seq + n))
        for t in (k, v, q):
            t.copy_(torch.randn_like(t))
        g.replay()
        b.step()
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and torch.equal(a.table, b.table), i
        assert all(torch.equal(x, y) for x, y in zip(a.lay, b.lay)), i
        assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.pool.free, b.pool.free), i
        seq += n
