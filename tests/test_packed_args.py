"""What the calls of packed batches refuse beyond single arguments: memory that is shared, sizes at the
end of their range, a pool's buffers exchanged (CPU: addresses are compared, never read)."""
import ctypes

import pytest

import suffix_match_drafter_amd as sfx


def ptr(x):
    return None if x is None else ctypes.c_void_p(x)


def error():
    return sfx.load().sfx_last_error().decode()


# ------------------------------------------------------------------ the layout
LAYOUT = dict(table=1 << 20, start=2 << 20, count=3 << 20, offsets=4 << 20, seq_lens=5 << 20,
              request=6 << 20, position=7 << 20, slots=8 << 20)


def layout(B=10, N=100, mp=3, **at):
    a = dict(LAYOUT, **at)
    return sfx.load().sfx_step_layout(B, N, mp, 64, 30, *(ptr(a[n]) for n in LAYOUT), None)


@pytest.mark.parametrize("out", ["offsets", "seq_lens", "request", "position", "slots"])
@pytest.mark.parametrize("other", ["table", "start", "count", "seq_lens", "request", "slots"])
def test_layout_refuses_shared_memory(out, other):
    """The same array twice, and two that meet in one element."""
    if out == other:
        return
    size = dict(table=120, start=40, count=40, offsets=44, seq_lens=40, request=400, position=400,
                slots=800)
    for at in (LAYOUT[other], LAYOUT[other] + size[other] - 4, LAYOUT[other] - size[out] + 4):
        assert layout(**{out: at}) == sfx.EINVAL, at
        assert "share memory" in error()


def test_layout_takes_neighbours():
    """Arrays right behind each other, and no table beside a call without slots, are not refused for
    it: such a call ends at the launch, of which the CPU knows nothing."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the call would run")
    at = LAYOUT["start"]
    for kw in (dict(seq_lens=at + 40), dict(seq_lens=at - 40), dict(slots=at + 40),
               dict(slots=None, request=LAYOUT["table"])):
        assert layout(**kw) not in (sfx.OK, sfx.EINVAL, sfx.ECAPACITY), kw


# ------------------------------------------------------------------ the pool
@pytest.mark.parametrize("name", ["free", "num_free", "num_pages", "page_size", "device", "_index",
                                  "_bytes"])
def test_a_pool_keeps_its_buffers(name):
    """reserve hands their addresses and sizes on unchecked: another list would be written past its
    end, or misread."""
    pool = sfx.PagePool(8, 64, device="cpu")
    was = getattr(pool, name)
    with pytest.raises(AttributeError, match=name):
        setattr(pool, name, was)
    with pytest.raises(AttributeError, match=name):
        delattr(pool, name)
    assert getattr(pool, name) is was
    pool.note = "other attributes are the caller's"
    pool.note = "and can change"


RESERVE = dict(tokens=1 << 20, table=2 << 20, held=3 << 20, free=4 << 20, num_free=5 << 20,
               missing=6 << 20, ws=7 << 20)


def reserve(B=10, mp=3, pages=30, nws=1 << 18, **at):
    a = dict(RESERVE, **at)
    return sfx.load().sfx_pages_reserve(B, mp, 64, pages, *(ptr(a[n]) for n in RESERVE), nws, None)


@pytest.mark.parametrize("B,mp", [(10, 3), (5000, 3)])
@pytest.mark.parametrize("one", ["table", "held", "free", "num_free", "missing", "ws"])
@pytest.mark.parametrize("other", list(RESERVE))
def test_reserve_refuses_shared_memory(one, other, B, mp):
    """The same array twice, and two that meet in one element."""
    size = dict(tokens=4 * B, table=4 * B * mp, held=4 * B, free=120, num_free=4, missing=4 * B,
                ws=16 + 12 * B)
    if one == other or ("ws" in (one, other) and B <= 4096):   # small calls use no workspace
        return
    at = [RESERVE[other], RESERVE[other] + size[other] - 4, RESERVE[other] - size[one] + 4]
    if (one, other) == ("missing", "tokens"):
        at = at[1:]   # the very same array is not refused: see below
    for x in at:
        if one == "ws" and x % 16:
            continue
        assert reserve(B, mp, **{one: x}) == sfx.EINVAL, x
        assert "share memory" in error()


def test_reserve_takes_neighbours():
    """Arrays right behind each other, and missing in the place of tokens, end at the launch only."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the call would run")
    for kw in (dict(held=RESERVE["tokens"] + 40), dict(num_free=RESERVE["free"] + 120),
               dict(missing=RESERVE["tokens"]), dict(missing=None), dict(ws=RESERVE["table"])):
        assert reserve(**kw) not in (sfx.OK, sfx.EINVAL, sfx.ECAPACITY), kw


# ------------------------------------------------------------------ sizes at the end of their range
@pytest.mark.parametrize("B", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_as_many_requests_as_an_int_holds(B):
    """Workgroups count requests in steps of 1024, which has to end below 2^31."""
    far = {n: (i + 1) << 40 for i, n in enumerate(LAYOUT)}
    assert layout(B=B, mp=1, **far) == sfx.ECAPACITY
    assert "too large" in error()
    far = {n: (i + 1) << 40 for i, n in enumerate(RESERVE)}
    for mp in (0, 1):
        assert reserve(B=B, mp=mp, nws=1 << 39, **far) == sfx.ECAPACITY
        n = ctypes.c_size_t()
        size = sfx.load().sfx_pages_reserve_workspace_bytes
        assert size(B, mp, ctypes.byref(n)) == sfx.ECAPACITY
        assert size(2 ** 31 - 1024, mp, ctypes.byref(n)) == sfx.OK and n.value > 3 * 4 * (2 ** 31 - 1024)


# ------------------------------------------------------------------ attention
I64x2 = ctypes.c_int64 * 2
ROWS = dict(q=1 << 30, k=2 << 30, v=3 << 30, out=4 << 30)


def prompt(N=50, H=4, Hk=2, D=64, qs=None, ks=None, vs=None, **at):
    a = dict(ROWS, **at)
    strides = [None if s is None else I64x2(*s) for s in (qs, ks, vs)]
    return sfx.load().sfx_prompt_attention(2, N, H, Hk, D, ptr(5 << 30), ptr(a["q"]), strides[0],
                                           ptr(a["k"]), strides[1], ptr(a["v"]), strides[2],
                                           ptr(a["out"]), 0, 0.1, 0, 0, ptr(6 << 30), 1 << 30, None)


def packed(N=50, H=4, max_q=50, qs=None, **at):
    a = dict(ROWS, **at)
    c = sfx._KvCache(4, 64, 2, 64, 10 << 30, 11 << 30, 12 << 30, 13 << 30)
    return sfx.load().sfx_kv_attention_packed(
        ctypes.byref(c), 2, N, max_q, H, 2, ptr(5 << 30), ptr(7 << 30), ptr(8 << 30), ptr(a["q"]),
        None if qs is None else I64x2(*qs), ptr(a["out"]), 0, 0.1, 0, 0, ptr(6 << 30), 1 << 30, None)


def test_attention_refuses_outputs_over_its_inputs():
    """Rows are stored while other workgroups still read keys, values and (unless a row's result takes
    its query's own place) queries."""
    row = 4 * 64 * 2
    for name, size in (("k", 50 * row // 2), ("v", 50 * row // 2)):
        for at in (ROWS[name], ROWS[name] + size - 16, ROWS[name] - 50 * row + 16):
            assert prompt(out=at) == sfx.EINVAL and f"out and {name} share" in error()
    for call in (prompt, packed):
        for at in (ROWS["q"] + 16, ROWS["q"] + row, ROWS["q"] - row, ROWS["q"] + 49 * row):
            assert call(out=at) == sfx.EINVAL and "out and q share" in error(), at
        # the first of two tokens' rows fits its place, the second does not; heads in another order
        assert call(out=ROWS["q"], qs=(2 * 256, 64)) == sfx.EINVAL
        assert call(out=ROWS["q"], qs=(64, 50 * 64)) == sfx.EINVAL
        assert call(out=ROWS["q"], qs=(0, 64)) == sfx.EINVAL
    # between the first token's keys and the second's is room for 2 rows of out and no more
    gap = ROWS["k"] + row // 2
    assert prompt(N=2, out=gap, ks=(128 + 512 - 8, 64)) == sfx.EINVAL


def test_attention_takes_outputs_beside_its_inputs():
    """Dense queries may be replaced by their results, and outputs may lie between the rows of the inputs
    as long as they meet none of them: such calls end at the launch only."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("the call would run")
    row = 4 * 64 * 2
    ok = [prompt(out=ROWS["q"]), packed(out=ROWS["q"]), prompt(out=ROWS["q"], qs=(256, 64)),
          packed(N=1, max_q=1, out=ROWS["q"], qs=(9999, 64)), prompt(out=ROWS["k"] + 50 * row // 2),
          prompt(out=ROWS["v"] - 50 * row), packed(out=ROWS["q"] + 50 * row),
          prompt(N=2, out=ROWS["k"] + row // 2, ks=(128 + 512, 64)),
          prompt(N=2, out=ROWS["q"] + row, qs=(768, 64)),
          # heads far apart, the outputs between them
          prompt(out=ROWS["q"] + 50 * 128, qs=(64, 1 << 20))]
    assert all(rc not in (sfx.OK, sfx.EINVAL, sfx.ECAPACITY) for rc in ok), ok
