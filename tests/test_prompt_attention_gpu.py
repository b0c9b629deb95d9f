"""Attention of packed whole prompts against the definition in 64 bits.

Tolerance of one output o = sum p v, from the kernel's roundings:
  the result's own rounding, eps/2 of |o|;
  each weight p rounded to the values' type, eps/2 of it (fp16: below 2^-22 of the largest weight
  to a multiple of 2^-33 of it at worst, once per token);
  a score's fp32 error: (dim + 8) 2^-24 of sum |q||k| scale plus its own size, twice (numerator
  and denominator), as a relative error of the weights;
  fp32 sums: one rounding of 2^-23 per 16 tokens, 64 more in and after the matrix product;
all but the first in units of A = sum p |v|."""
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


def make(rng, n, heads, group, dim, dtype, fused=True):
    """q, k, v as views of one projection's output, or dense."""
    import torch

    x = torch.from_numpy(rng.standard_normal((n, heads * (group + 2), dim))).cuda()
    x = x.to(getattr(torch, dtype))
    parts = x.split((heads * group, heads, heads), 1)
    return parts if fused else tuple(p.contiguous() for p in parts)


def compare(got, q, k, v, offsets, window=0, sinks=0, scale=None, only=None):
    import torch

    eps = torch.finfo(got.dtype).eps / 2
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    out, q, k, v = (t.double().cpu().numpy() for t in (got, q, k, v))
    covered = np.zeros(len(out), bool)
    for b in range(len(offsets) - 1):
        lo, hi = offsets[b], offsets[b + 1]
        covered[lo:hi] = True
        if hi <= lo or (only is not None and b not in only):
            continue
        ref, mag, dots = M.prompt(q[lo:hi], k[lo:hi], v[lo:hi], scale, window, sinks)
        n = hi - lo
        rel = eps + 2 * (dim + 8) * 2.0 ** -24 * (dots + 1)[:, :, None] + \
            (n / 16 + 64) * 2.0 ** -23
        tol = eps * np.abs(ref) + mag * rel + n * 2.0 ** -33 * np.abs(v[lo:hi]).max()
        assert np.isfinite(out[lo:hi]).all(), b
        err = np.abs(out[lo:hi] - ref)
        assert (err <= tol).all(), (b, np.argwhere(err > tol)[:4], err.max(), tol.min())
    assert (out[~covered] == 0).all()


CASES = [
    # lens, heads, group, dim, window, sinks
    ([1], 1, 1, 64, 0, 0),
    ([1, 1, 1], 2, 4, 128, 0, 0),
    ([2, 0, 33], 2, 2, 64, 0, 0),
    ([31, 32, 33, 63, 64, 65], 1, 1, 128, 0, 0),
    ([127, 128, 129], 2, 3, 64, 0, 0),
    ([5, 300], 1, 5, 256, 0, 0),
    ([70, 1, 17], 2, 16, 256, 0, 0),
    ([400], 1, 1, 128, 0, 0),
    ([257, 3], 1, 8, 128, 0, 0),
    ([10] * 40, 2, 7, 64, 0, 0),
    ([200, 90], 1, 2, 128, 1, 0),
    ([200, 90], 1, 2, 128, 100, 0),
    ([300, 90], 1, 2, 128, 33, 4),
    ([300, 40], 1, 4, 64, 64, 100),
    ([300], 2, 2, 256, 5, 70),
    ([150], 1, 1, 64, 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_model(S, case, dtype):
    lens, heads, group, dim, window, sinks = case
    rng = np.random.default_rng(sum(lens) + dim)
    offsets = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = make(rng, offsets[-1], heads, group, dim, dtype)
    out = S.attend_prompt(q, k, v, i32(offsets), window=window, sinks=sinks)
    compare(out, q, k, v, offsets, window, sinks)


@pytest.mark.parametrize("B", [61, 62, 63, 64, 65, 300, 5000])
def test_many_requests(S, B):
    """Requests of no to a few rows, found by one, two or three rounds of probes."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 4, B)
    lens[B // 2] = 150
    offsets = np.concatenate([[0], np.cumsum(lens)]) + 5
    q, k, v = make(rng, int(offsets[-1]) + 9, 1, 3, 64, "float16")
    out = S.attend_prompt(q, k, v, i32(offsets))
    compare(out, q, k, v, offsets)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_split_by_tokens(S, dim):
    """Few rows, many tokens: parts of one row tile joined (some tiles have one part only)."""
    rng = np.random.default_rng(dim)
    offsets = [0, 5, 1300, 1301]
    q, k, v = make(rng, 1301, 1, 1, dim, "float16", fused=False)
    for window, sinks in ((0, 0), (700, 3)):
        out = S.attend_prompt(q, k, v, i32(offsets), window=window, sinks=sinks)
        compare(out, q, k, v, offsets, window, sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_of_no_request(S, dim):
    """Rows before the first request, between none and behind the last hold NaN: nobody sees them and
    their results are zero.  Offsets past the rows are cut."""
    import torch

    rng = np.random.default_rng(dim)
    q, k, v = make(rng, 700, 2, 2, dim, "bfloat16")
    offsets = [70, 100, 100, 350]
    for t in (q, k, v):
        t[:70] = float("nan")
        t[350:] = float("nan")
    out = S.attend_prompt(q, k, v, i32(offsets))
    compare(out, q, k, v, offsets)
    out = S.attend_prompt(q[:350], k[:350], v[:350], i32([70, 100, 100, 9999]))
    compare(out, q[:350], k[:350], v[:350], offsets)
    out = S.attend_prompt(q[:5], k[:5], v[:5], i32([0]))
    assert out.eq(0).all()
    out = S.attend_prompt(q[:0], k[:0], v[:0], i32([0, 0]))
    assert out.shape == (0, 4, dim)


@pytest.mark.parametrize("special", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,dim", [("bfloat16", 128), ("float16", 64), ("bfloat16", 256)])
def test_special_values_reach_their_rows_only(S, dtype, dim, special):
    """One infinite or NaN value: the rows that do not see it (before it, past the window, of other
    requests) are as without it, the others have it in that dim and nothing else."""
    import torch

    rng = np.random.default_rng(3)
    offsets, at, window, sinks = [0, 60, 400], 60 + 133, 90, 2
    q, k, v = make(rng, 400, 1, 2, dim, dtype, fused=False)
    plain = S.attend_prompt(q, k, v, i32(offsets), window=window, sinks=sinks)
    v[at, 0, 5] = special
    v[60 + 1, 0, 9] = special   # a sink: everything after it
    out = S.attend_prompt(q, k, v, i32(offsets), window=window, sinks=sinks)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[at:at + window, :, 5] = True
    hit[61:400, :, 9] = True
    assert torch.equal(out[~hit], plain[~hit])
    got = out[hit]
    assert (got.isnan() if special != special else got == special).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_keys_that_are_not_seen(S, dim):
    """NaN and infinite keys of later rows change nothing before them; a row that sees a NaN key is
    NaN, one that sees a key of -inf score leaves it out."""
    import torch

    rng = np.random.default_rng(4)
    q, k, v = make(rng, 300, 1, 1, dim, "float16", fused=False)
    q[:, :, 0] = 1.0
    plain = S.attend_prompt(q, k, v, i32([0, 300]))
    bad = k.clone()
    bad[200, 0, 3] = float("nan")
    out = S.attend_prompt(q, bad, v, i32([0, 300]))
    assert torch.equal(out[:200], plain[:200]) and out[200:].isnan().all()
    bad = k.clone()
    bad[200] = 0
    bad[200, 0, 0] = float("-inf")
    out = S.attend_prompt(q, bad, v, i32([0, 300]))
    assert torch.equal(out[:200], plain[:200]) and out.isfinite().all()
    # alone with a score of -inf: nothing to see
    out = S.attend_prompt(q[200:201], bad[200:201], v[200:201], i32([0, 1]))
    assert out.eq(0).all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("scale", [2.0 ** -40, 30.0, 2.0 ** 22])
def test_scales(S, dtype, scale):
    """Even weights and weights of one token alone; scores up to 2^31 that differ exactly."""
    rng = np.random.default_rng(5)
    import torch

    n, dim = 200, 64
    q, k, v = make(rng, n, 1, 2, dim, dtype, fused=False)
    if scale > 2:
        # small whole numbers: products and sums are exact in fp32
        q.copy_(torch.from_numpy(rng.integers(-2, 3, q.shape)))
        k.copy_(torch.from_numpy(rng.integers(-2, 3, k.shape)))
    out = S.attend_prompt(q, k, v, i32([0, n]), scale=scale)
    qq, kk, vv = (t.double().cpu().numpy() for t in (q, k, v))
    if scale < 2:
        compare(out, q, k, v, [0, n], scale=scale)
        return
    ref, mag, _ = M.prompt(qq, kk, vv, scale, 0, 0)
    # scores are whole multiples of the scale, at least 30 apart or equal: weights are 1 / m or
    # below e^-30, whose rounding adds nothing
    eps = torch.finfo(out.dtype).eps / 2
    tol = eps * np.abs(ref) + mag * (eps + 2.0 ** -16) + n * np.exp(-29.0) * np.abs(vv).max()
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


def test_strides(S):
    """Odd row and head strides, heads before rows, one key head shared by expansion."""
    import torch

    rng = np.random.default_rng(6)
    n, dim = 130, 64
    want_q, want_k, want_v = make(rng, n, 2, 2, dim, "bfloat16", fused=False)
    want = S.attend_prompt(want_q, want_k, want_v, i32([0, 50, n]))

    def odd(t, extra):
        wide = torch.full((t.shape[0], t.shape[1], t.shape[2] + extra), float("nan"),
                          dtype=t.dtype, device="cuda")
        wide[:, :, 1:dim + 1] = t
        return wide[:, :, 1:dim + 1]

    for args in ((odd(want_q, 3), odd(want_k, 5), odd(want_v, 7)),
                 tuple(t.transpose(0, 1).contiguous().transpose(0, 1)
                       for t in (want_q, want_k, want_v))):
        assert not args[0].is_contiguous()
        assert torch.equal(S.attend_prompt(*args, i32([0, 50, n])), want)
    # rows 32 MB apart
    far = torch.empty((2 ** 24 + 8) * (n - 1) + 8 * dim, dtype=torch.bfloat16, device="cuda")
    parts = []
    for t, at in ((want_q, 0), (want_k, 4 * dim), (want_v, 6 * dim)):
        parts.append(far.as_strided(t.shape, (2 ** 24 + 8, dim, 1), at))
        parts[-1].copy_(t)
    assert torch.equal(S.attend_prompt(*parts, i32([0, 50, n])), want)
    one_k, one_v = want_k[:, :1].expand(n, 2, dim), want_v[:, :1].expand(n, 2, dim)
    shared = S.attend_prompt(want_q, one_k, one_v, i32([0, 50, n]))
    dense = S.attend_prompt(want_q, one_k.contiguous(), one_v.contiguous(), i32([0, 50, n]))
    assert torch.equal(shared, dense)


def test_graph_and_streams(S):
    """Captured once, replayed with other lengths and inputs, each time as the eager call."""
    import torch

    rng = np.random.default_rng(7)
    n, dim = 900, 128
    q, k, v = make(rng, n, 1, 4, dim, "bfloat16", fused=False)
    offsets = i32([0, 300, 900])
    out = torch.empty_like(q)
    S.attend_prompt(q, k, v, offsets, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.attend_prompt(q, k, v, offsets, out=out)
    for i, off in enumerate(([0, 1, 900], [0, 900, 900], [4, 5, 6], [0, 300, 899])):
        offsets.copy_(i32(off))
        q.copy_(torch.randn_like(q))
        v.copy_(torch.randn_like(v))
        out.fill_(7)
        g.replay()
        got = out.clone()
        assert torch.equal(got, S.attend_prompt(q, k, v, offsets)), i
        torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = S.attend_prompt(q, k, v, offsets, stream=st)
    st.synchronize()
    assert torch.equal(got, S.attend_prompt(q, k, v, offsets))


def test_long_prompt(S):
    """Sampled rows of a prompt of 5000 tokens."""
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n, dim = 5000, 128
    q, k, v = (torch.randn((n, h, dim), generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    out = S.attend_prompt(q, k, v, i32([0, n])).double().cpu().numpy()
    kk, vv = k.double().cpu().numpy(), v.double().cpu().numpy()
    for t in (0, 1, 63, 64, 1000, 2047, 2048, 4095, 4999):
        for h in range(4):
            s = kk[:t + 1, h // 2] @ q[t, h].double().cpu().numpy() * dim ** -0.5
            w = np.exp(s - s.max())
            w /= w.sum()
            ref, mag = w @ vv[:t + 1, h // 2], w @ np.abs(vv[:t + 1, h // 2])
            tol = 2.0 ** -8 * np.abs(ref) + mag * (2.0 ** -8 + 400 * 2.0 ** -23 +
                                                   2 * (dim + 8) * 2.0 ** -24 * 40)
            assert (np.abs(out[t, h] - ref) <= tol).all(), (t, h)
