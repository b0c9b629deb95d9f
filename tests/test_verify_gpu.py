"""Draft verification against the model in 64 bits (tests/kv_model.py): tokens and counts are
compared exactly."""
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


def case(rng, B, k, V, dtype, take=0.6):
    """Logits [B, k + 1, V] in `dtype`, drafts that the target likes with chance `take`."""
    import torch

    x = rng.standard_normal((B, k + 1, V)) * 2
    draft = rng.integers(0, V, size=(B, k)).astype(np.int32)
    like = rng.random((B, k)) < take
    for b in range(B):
        for i in range(k):
            if like[b, i]:
                x[b, i, draft[b, i]] = np.log(V) + 3
    t = torch.from_numpy(x).to(getattr(torch, dtype))
    return t.cuda(), draft, rng.integers(0, k + 1, size=B).astype(np.int32), \
        rng.random((B, k)).astype(np.float32), rng.random(B).astype(np.float32), \
        rng.uniform(0.3, 2.0, B).astype(np.float32)


def check(S, logits, draft, nv, ua, us, temp):
    import torch

    out, na = S.verify(logits, dev(draft), None if nv is None else dev(nv), dev(ua), dev(us),
                       None if temp is None else dev(temp))
    torch.cuda.synchronize()
    x = logits.double().cpu().numpy()
    B, k1 = x.shape[:2]
    for b in range(B):
        s, n = M.verify(x[b], draft[b], k1 - 1 if nv is None else nv[b], ua[b], us[b],
                        1.0 if temp is None else float(temp[b]))
        assert na[b].item() == n and np.array_equal(out[b].cpu().numpy(), s), \
            (b, out[b].tolist(), s, na[b].item(), n)
    return out, na


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("B,k,V", [(1, 1, 1), (3, 2, 2), (5, 4, 7), (8, 8, 1000), (4, 32, 513),
                                   (16, 3, 4099), (2, 16, 40001), (1, 5, 151936)])
def test_against_model(S, B, k, V, dtype):
    rng = np.random.default_rng(B * 100 + V)
    check(S, *case(rng, B, k, V, dtype))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_greedy(S, dtype):
    """T = 0, below 0 and NaN; ties go to the lowest index, also across the row's parts."""
    rng = np.random.default_rng(1)
    x, draft, nv, ua, us, temp = case(rng, 8, 4, 40000, dtype)
    temp[:] = [0.0, -1.0, np.nan, -np.inf, 0.0, 0.0, 1.0, -0.0]
    x[4, :, 39990] = 50.0
    x[4, :, 17] = 50.0
    x[5, 0] = 1.0
    draft[5, 0], nv[5] = 0, 4
    check(S, x, draft, nv, ua, us, temp)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_masked_logits(S, dtype):
    """-inf and the type's lowest value as masks, NaN, +inf, rows that leave nothing or one."""
    import torch

    rng = np.random.default_rng(2)
    x, draft, nv, ua, us, temp = case(rng, 12, 3, 300, dtype)
    low = torch.finfo(x.dtype).min
    nv[:] = 3
    x[0, :, 50:] = -float("inf")
    x[1, :, 50:] = low
    x[2] = -float("inf")
    x[3] = float("nan")
    x[4, :, 5] = float("nan")
    x[5, 0, [7, 9]] = float("inf")
    draft[5, 0] = 9
    x[6] = -float("inf")
    x[6, :, 123] = 0.0
    draft[6] = [123, 5, 123]
    x[7] = low
    x[8] = 1.0
    x[9, 0, :] = float("inf")
    temp[8:10] = [np.inf, 1e-30]
    x[10] = -float("inf")
    x[10, :, 40] = 3.0
    draft[10] = [40, 40, 40]
    temp[10] = 0.0
    x[11] = float("nan")
    temp[11] = 0.0
    check(S, x, draft, nv, ua, us, temp)
    temp[:] = np.inf
    check(S, x, draft, nv, ua, us, temp)
    temp[:] = np.float32(1e-42)
    check(S, x, draft, nv, ua, us, temp)


def test_borders(S):
    """Tests and draws whose two sides are equal in exact arithmetic, or one float apart."""
    import torch

    V, k, B = 8, 2, 64
    x = torch.zeros((B, k + 1, V), device="cuda")       # every weight is exactly 1
    draft = np.tile(np.arange(2, dtype=np.int32), (B, 1))
    nv = np.full(B, k, np.int32)
    ua, us = np.zeros((B, k), np.float32), np.zeros(B, np.float32)
    eighth = np.float32(0.125)
    ua[:16] = eighth                                     # u Z = w: not accepted
    ua[16:32] = np.nextafter(eighth, np.float32(0))      # accepted
    ua[32:48] = np.nextafter(eighth, np.float32(1))
    for b in range(B):
        # running sums of 7 (a rejected draft) or 8 equal weights: their borders exactly
        us[b] = np.float32(b % 8) * eighth
    us[-1] = np.nextafter(np.float32(1), np.float32(0))
    check(S, x, draft, nv, ua, us, None)
    check(S, x, draft, None, ua, us, np.full(B, 0.7, np.float32))


def test_drafts_outside_the_vocabulary(S):
    rng = np.random.default_rng(3)
    x, draft, nv, ua, us, temp = case(rng, 6, 3, 100, "float32")
    nv[:] = [3, 3, 3, 7, -2, 0]
    draft[0, 0], draft[1, 0], draft[2, 1] = -1, 100, 2 ** 31 - 1
    draft[3] = -2 ** 31
    ua[:] = 0.0
    check(S, x, draft, nv, ua, us, temp)
    temp[:] = 0.0
    check(S, x, draft, nv, ua, us, temp)


def test_flat_and_peaked_rows(S):
    """Draws along a flat large row (every border is within a float's rounding of the next) and
    from rows with one heavy token; all random numbers, 0 and the largest below 1."""
    import torch

    V, B = 100003, 48
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((B, 1, V), generator=g, device="cuda") * 0.01
    x[24:, :, 77777] = 14.0
    us = np.linspace(0, 1, B, endpoint=False).astype(np.float32)
    us[23] = us[47] = np.nextafter(np.float32(1), np.float32(0))
    empty = np.zeros((B, 0), np.int32)
    check(S, x, empty, None, empty.astype(np.float32), us, None)
    check(S, x.to(torch.bfloat16), empty, np.full(B, 5, np.int32), empty.astype(np.float32), us,
          np.full(B, 0.8, np.float32))


def test_strides_and_outputs(S):
    """Rows of a wider buffer at odd offsets; given outputs; nothing past num_valid is read."""
    import torch

    rng = np.random.default_rng(5)
    B, k, V = 5, 6, 1001
    x, draft, nv, ua, us, temp = case(rng, B, k, V, "bfloat16")
    wide = torch.full((k + 1, B, V + 7), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = wide[:, :, 3:3 + V].transpose(0, 1)
    view.copy_(x)
    a = check(S, view, draft, nv, ua, us, temp)
    out = torch.full((B, k + 1), 9, dtype=torch.int32, device="cuda")
    na = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    got = S.verify(x, dev(draft), dev(nv), dev(ua), dev(us), dev(temp), sampled=out,
                   num_accepted=na)
    assert got[0] is out and got[1] is na
    assert torch.equal(out, a[0]) and torch.equal(na, a[1])
    for b in range(B):
        x[b, nv[b] + 1:] = float("inf")
    assert torch.equal(S.verify(x, dev(draft), dev(nv), dev(ua), dev(us), dev(temp))[0], out)
    assert S.verify(x[:0], dev(draft)[:0], None, dev(ua)[:0], dev(us)[:0])[0].shape == (0, k + 1)


def test_graph_and_stream(S):
    import torch

    rng = np.random.default_rng(6)
    B, k, V = 7, 4, 30011
    x, draft, nv, ua, us, temp = case(rng, B, k, V, "float16")
    bufs = [x.clone(), dev(draft), dev(nv), dev(ua), dev(us), dev(temp)]
    out = torch.empty((B, k + 1), dtype=torch.int32, device="cuda")
    na = torch.empty((B,), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        S.verify(*bufs, sampled=out, num_accepted=na, stream=s)
    for step in range(4):
        new = case(rng, B, k, V, "float16")
        for b, n in zip(bufs, new):
            b.copy_(n if isinstance(n, torch.Tensor) else dev(n))
        out.fill_(-7)
        g.replay()
        want = check(S, *new)
        assert torch.equal(out, want[0]) and torch.equal(na, want[1]), step
        s.wait_stream(torch.cuda.current_stream())
        mine = S.verify(*bufs, stream=s)
        s.synchronize()
        assert torch.equal(mine[0], want[0]) and torch.equal(mine[1], want[1])


def test_step_with_the_drafter(S):
    """propose -> verify -> feedback and update: the verifier's outputs are the drafter's next
    inputs, and a greedy target that repeats the draft accepts all of it."""
    import torch

    rng = np.random.default_rng(8)
    B, Sq, V, k = 4, 64, 50, 8
    d = S.Drafter(S.Config(k=k, max_tree_depth=8, max_batch=B, max_seq=Sq, max_sampled=k + 1))
    period = rng.integers(0, V, size=(B, 5)).astype(np.int32)
    tok = dev(np.tile(period, (1, 13))[:, :Sq])
    n = dev(np.full(B, 20, np.int32))
    samp = torch.full((B, k + 1), -1, dtype=torch.int32, device="cuda")
    samp[:, 0] = tok[:, 20]
    draft, nv = d.propose(n, tok, samp)
    logits = torch.zeros((B, k + 1, V), device="cuda")
    want = torch.from_numpy(np.tile(period, (1, 13))[:, 21:21 + k + 1]).cuda()
    logits.scatter_(2, want.long()[:, :, None], 5.0)
    zero = torch.zeros((B,), device="cuda")
    out, na = S.verify(logits, draft, nv, torch.zeros((B, k), device="cuda"), zero, zero)
    assert na.tolist() == nv.tolist() == [k] * B and torch.equal(out, want)
    d.accept_feedback(na)
    after = S.update_state(tok.clone(), S.update_state(tok, n, samp), out)
    assert after.tolist() == [21 + k + 1] * B
    d.close()


@pytest.mark.parametrize("dtype,B,k,V", [("float32", 26, 16, 120011), ("bfloat16", 150, 32, 20481),
                                         ("float16", 2048, 3, 12345), ("float16", 2049, 3, 12345)])
def test_large_calls(S, dtype, B, k, V):
    """Calls large enough to go through the slots in phases (and one too wide for that): all
    accepted, none, greedy, masked rows, counts of 0 and k, and a second pass over one workspace's
    worth of memory."""
    rng = np.random.default_rng(V)
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.randn((B, k + 1, V), generator=g, device="cuda").mul_(2).to(getattr(torch, dtype))
    draft = rng.integers(0, V, size=(B, k)).astype(np.int32)
    nv = rng.integers(0, k + 1, size=B).astype(np.int32)
    like = rng.random((B, k)) < 0.85
    like[:4] = True
    nv[:4] = k
    like[4:8] = False
    at = np.where(like, draft, rng.integers(0, V, size=(B, k)))
    x[:, :k].scatter_(2, dev(at)[:, :, None], 16.0)
    temp = rng.uniform(0.5, 1.3, B).astype(np.float32)
    temp[[1, 5, 9, 10]] = 0.0
    ua = rng.random((B, k)).astype(np.float32)
    us = rng.random(B).astype(np.float32)
    ua[0] = 0.0
    x[11, 0] = -float("inf")
    x[12, 1, ::2] = -float("inf")
    x[13, 0, 5] = float("nan")
    x[14, 0, [7, V - 1]] = float("inf")
    nv[11:15] = k
    rows = list(range(15)) + list(range(15, B, max(1, B // 12)))
    for step in range(2):
        out, na = S.verify(x, dev(draft), dev(nv), dev(ua), dev(us), dev(temp))
        torch.cuda.synchronize()
        for b in rows:
            s, n = M.verify(x[b].double().cpu().numpy(), draft[b], nv[b], ua[b], us[b],
                            float(temp[b]))
            assert na[b].item() == n and np.array_equal(out[b].cpu().numpy(), s), (b, n)
        us = rng.random(B).astype(np.float32)
        ua = rng.random((B, k)).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,V", [(1, 4097), (1, 8192), (2, 70001), (3, 262147), (20, 33000),
                                 (100, 9001), (129, 9001), (2, 4096), (2, 1025), (2, 1024)])
def test_draws(S, dtype, B, V):
    """Draws alone, over every way of splitting a row: first and last tokens, u of 0, masked ends,
    heavy tokens at the borders of segments."""
    import torch

    rng = np.random.default_rng(V)
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    x = torch.randn((B, 1, V), generator=g, device="cuda").to(getattr(torch, dtype))
    empty = np.zeros((B, 0), np.int32)
    for step in range(6):
        us = rng.random(B).astype(np.float32)
        if step == 1:
            us[:] = 0.0
        if step == 2:
            us[:] = np.nextafter(np.float32(1), np.float32(0))
        if step == 3:
            x[:, 0, :V // 3] = -float("inf")
            us[0] = 0.0
        if step == 4:
            x[:, 0, V - V // 5:] = -float("inf")
            us[:] = np.nextafter(np.float32(1), np.float32(0))
        if step == 5:
            for j in (V // 2, V // 2 + 1, V // 16 * 9, V // 16 * 9 - 1):
                x[:, 0, j] = 11.0
        check(S, x, empty, None, empty.astype(np.float32), us, None)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("V", [300, 1024, 5000, 40001])
@pytest.mark.parametrize("temp", [0.0, 1e-30, 1.0, 1e31, 1e38, np.inf])
def test_infinite_logits_share_the_row(S, dtype, V, temp):
    """Logits of +inf leave nothing to finite ones, the type's largest value among them, whatever
    the temperature; greedy takes the first +inf.  A draft among n of them has weight 1 / n."""
    import torch

    rng = np.random.default_rng(V)
    B, k, n = 16, 2, 4
    x = rng.standard_normal((B, k + 1, V))
    x = torch.from_numpy(x).to(getattr(torch, dtype)).cuda()
    x[:, :, ::3] = torch.finfo(x.dtype).max
    x[3, :, 1::3] = -float("inf")
    x[5, :, 1::3] = float("nan")
    draft = np.zeros((B, k), np.int32)
    for b in range(B):
        for i in range(k + 1):
            at = rng.choice(np.arange(1, V), n, replace=False)
            x[b, i, dev(at)] = float("inf")
            if i < k:
                draft[b, i] = np.sort(at)[0 if b % 4 == 0 else rng.integers(0, n)]
    draft[15, 0] = 0  # finite
    ua = np.full((B, k), 0.3, np.float32)
    ua[:8] = np.nextafter(np.float32(0.25), np.float32(0))
    ua[8:12, 1] = 0.25
    us = rng.random(B).astype(np.float32)
    us[0], us[1] = 0.0, np.nextafter(np.float32(1), np.float32(0))
    check(S, x, draft, None, ua, us, np.full(B, temp, np.float32))


@pytest.mark.parametrize("temp", [1.0, np.inf])
def test_infinite_logits_in_phases(S, temp):
    """The same in a call that goes through the slots in phases."""
    import torch

    rng = np.random.default_rng(9)
    B, k, V = 26, 16, 120011
    x = torch.zeros((B, k + 1, V), device="cuda")
    x[:, :, ::7] = torch.finfo(x.dtype).max
    draft = rng.integers(2000, V // 2, size=(B, k)).astype(np.int32)
    for i in range(k + 1):
        at = draft[:, i] if i < k else np.full(B, 77, np.int32)
        for far in (0, -1500, 30011, 60000):
            x[dev(np.arange(B)), i, dev(at + far).long() % V] = float("inf")
    ua = np.full((B, k), np.nextafter(np.float32(0.25), np.float32(0)), np.float32)
    for b in range(B):
        ua[b, b:] = 0.25
    us = rng.random(B).astype(np.float32)
    check(S, x, draft, None, ua, us, np.full(B, temp, np.float32))


def masked_rows(rng, B, k, V, dtype):
    """Rows with 512 tokens left: masks of -inf or NaN in one run (so that whole segments of a row
    are masked) or scattered, and drafts among the tokens that are left."""
    import torch

    x = rng.standard_normal((B, k + 1, V))
    draft = np.zeros((B, k), np.int32)
    for b in range(B):
        for i in range(k + 1):
            first = rng.integers(0, V - 512)
            left = np.arange(first, first + 512) if b % 2 else rng.choice(V, 512, replace=False)
            out = np.ones(V, bool)
            out[left] = False
            x[b, i, out] = np.nan if b % 3 == 2 else -np.inf
            if i < k:
                draft[b, i] = left[rng.integers(0, 512)]
    return torch.from_numpy(x).to(getattr(torch, dtype)).cuda(), draft


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("V", [1025, 4096, 4097, 40001])
@pytest.mark.parametrize("temp", [1e31, 1e37, 1e38, np.inf])
def test_masks_at_large_temperatures(S, dtype, V, temp):
    """A masked token, and the draft that was rejected, weigh nothing at any temperature.  The 512
    tokens that are left have a weight of 1 each, so a draft is accepted just below u = 1 / 512."""
    rng = np.random.default_rng(V)
    border = np.float32(1 / 512)
    for k in (0, 3):
        B = 24
        x, draft = masked_rows(rng, B, k, V, dtype)
        ua = np.full((B, k), 0.75, np.float32)
        if k:
            ua[:8] = np.nextafter(border, np.float32(0))
            ua[8:12] = border
            ua[12:16, 0] = np.nextafter(border, np.float32(0))
        us = rng.random(B).astype(np.float32)
        us[0], us[1] = 0.0, np.nextafter(np.float32(1), np.float32(0))
        check(S, x, draft, None, ua, us, np.full(B, temp, np.float32))


@pytest.mark.parametrize("temp", [1e31, np.inf])
def test_masks_at_large_temperatures_in_phases(S, temp):
    """The same in a call that goes through the slots in phases."""
    import torch

    rng = np.random.default_rng(7)
    B, k, V = 26, 16, 120011
    x = torch.full((B, k + 1, V), -float("inf"), device="cuda")
    draft = rng.integers(512, V - 512, size=(B, k)).astype(np.int32)
    at = dev(draft.astype(np.int64))[:, :, None] + torch.arange(-256, 256, device="cuda")
    x[:, :k].scatter_(2, at, 0.5)
    x[:, k, 1000:1512] = -0.25
    border = np.float32(1 / 512)
    ua = np.full((B, k), np.nextafter(border, np.float32(0)), np.float32)
    for b in range(B):
        ua[b, b:] = border if b % 2 else 0.75
    us = rng.random(B).astype(np.float32)
    check(S, x, draft, None, ua, us, np.full(B, temp, np.float32))


@pytest.mark.parametrize("V", [1025, 5000, 40000])
def test_infinities_beside_the_lowest_float(S, V):
    """fp32 rows whose largest logit is the type's lowest value: -inf is masked all the same."""
    import torch

    rng = np.random.default_rng(V)
    B = 8
    x = torch.full((B, 1, V), -float("inf"), device="cuda")
    for b in range(B):
        x[b, 0, dev(rng.choice(V, 1 + 37 * b, replace=False))] = torch.finfo(torch.float32).min
    empty = np.zeros((B, 0), np.int32)
    us = rng.random(B).astype(np.float32)
    for temp in (1e-3, 1.0, 1e31):
        check(S, x, empty, None, empty.astype(np.float32), us, np.full(B, temp, np.float32))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("V", [300, 1025, 4097, 40001])
@pytest.mark.parametrize("temp", [1e29, 2e30, 1e31, 1e37, 1e38, 3e38, np.inf])
def test_finite_masks_at_large_temperatures(S, dtype, V, temp):
    """The type's lowest value is a logit like another: at a temperature as large as itself it has
    a weight, with which drafts are accepted and tokens drawn."""
    import torch

    rng = np.random.default_rng(V)
    B, k = 24, 3
    x, draft, nv, ua, us, _ = case(rng, B, k, V, dtype)
    nv[:] = k
    low = torch.finfo(x.dtype).min
    left = V // 3
    for b in range(B):
        x[b, :, left:] = low
        draft[b] = rng.integers(0, left if b % 3 else V, size=k)
        if b % 4 == 0:
            x[b, :, 2 * left:] = -float("inf")
        if b % 4 == 1:
            x[b, :, :left] = torch.finfo(x.dtype).max
    # about the weight of a masked and of another draft
    ua[:] = rng.choice([0.5, 0.9, 1.1, 2.0], (B, k)) / V
    check(S, x, draft, nv, ua, us, np.full(B, temp, np.float32))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [300, 5000, 40001])
@pytest.mark.parametrize("temp", [1e-29, 1e-30, 1e-31, 1e-35, 1e-38])
def test_small_temperatures_of_small_logits(S, dtype, V, temp):
    """Logits that differ by some temperatures, however small these are."""
    import torch

    rng = np.random.default_rng(V)
    B, k = 16, 3
    x = torch.from_numpy(rng.standard_normal((B, k + 1, V)) * 2 * max(temp, 1e-34))
    draft = rng.integers(0, V, size=(B, k)).astype(np.int32)
    at = torch.from_numpy(draft).long()[:, :, None]
    x[:, :k].scatter_(2, at, (np.log(V) + rng.uniform(-3, 3)) * temp)
    x = x.to(getattr(torch, dtype)).cuda()
    ua, us = rng.random((B, k)).astype(np.float32), rng.random(B).astype(np.float32)
    check(S, x, draft, None, ua, us, np.full(B, temp, np.float32))


@pytest.mark.parametrize("temp", [3e38, 1e-31])
def test_extreme_temperatures_in_phases(S, temp):
    """The same in a call that goes through the slots in phases."""
    import torch

    rng = np.random.default_rng(10)
    B, k, V = 26, 16, 120011
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    unit = 0.5 * temp
    x = torch.randn((B, k + 1, V), generator=g, device="cuda").clamp_(-1, 1) * unit
    draft = rng.integers(0, V, size=(B, k)).astype(np.int32)
    x[:, :k].scatter_(2, dev(draft).long()[:, :, None], unit * 1.5 if temp > 1 else unit * 24)
    ua = rng.random((B, k)).astype(np.float32) * (3.0 / V if temp > 1 else 1.0)
    us = rng.random(B).astype(np.float32)
    check(S, x, draft, None, ua.astype(np.float32), us, np.full(B, temp, np.float32))


def test_vocabulary_past_32_bits_is_refused(S):
    """2^32 + 5 logits a row would reach the library as 5."""
    import torch

    x = torch.empty((1, 1, 2 ** 32 + 5), dtype=torch.float16, device="cuda")
    none = torch.empty((1, 0), device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        S.verify(x, none.int(), None, none, torch.zeros(1, device="cuda"))
