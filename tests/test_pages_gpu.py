"""Pages handed out on the device and the layout of a packed batch, against the model: whole numbers,
equal everywhere that means something."""
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


class Both:
    """A pool on the device and the model's, step by step."""

    def __init__(self, S, rng, B, width, page, pages):
        import torch

        self.page, self.pages = page, pages
        self.free = rng.permutation(pages).astype(np.int32)
        self.nf = pages
        self.table = np.full((B, width), -1, np.int32)
        self.held = np.zeros(B, np.int32)
        self.pool = S.PagePool(pages, page, buffers=(i32(self.free), i32([pages])))
        self.d_table, self.d_held = i32(self.table), i32(self.held)
        self.torch = torch

    def step(self, tokens):
        missing = self.pool.reserve(self.d_table, self.d_held, i32(tokens))
        self.table, self.held, self.free, self.nf, want = M.reserve(
            self.table, self.held, self.free, self.nf, tokens, self.page, self.pages)
        assert missing.tolist() == want.tolist()
        self.check()
        return want

    def check(self):
        assert self.d_held.tolist() == self.held.tolist()
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert int(self.pool.num_free) == self.nf
        assert self.pool.free[:self.nf].tolist() == self.free[:self.nf].tolist()
        # every page is somewhere, once
        used = [int(p) for b, h in enumerate(self.held) for p in self.table[b, :h]]
        assert sorted(used + self.free[:self.nf].tolist()) == list(range(self.pages))


@pytest.mark.parametrize("B,width,page,pages", [
    (1, 1, 1, 1), (1, 5, 16, 3), (3, 4, 32, 9), (64, 9, 64, 400), (200, 81, 48, 5000),
    (1023, 12, 64, 9000), (1025, 3, 64, 2000), (4096, 4, 16, 9000), (4097, 4, 16, 9000),
    (300, 100, 1, 20000), (2500, 40, 7, 60000)])
def test_reserve(S, B, width, page, pages):
    """Growing, ending and new requests; now and then more than there is, or than a row holds."""
    rng = np.random.default_rng(B + width)
    both = Both(S, rng, B, width, page, pages)
    tokens = np.zeros(B, np.int64)
    lacked = 0
    for step in range(6):
        kind = rng.random(B)
        tokens = np.where(kind < 0.3, 0, np.where(kind < 0.6, rng.integers(0, width * page + 1, B),
                                                  np.minimum(tokens + rng.integers(0, 40, B),
                                                             width * page)))
        tokens[rng.random(B) < 0.02] = width * page + 1   # more than a row holds
        tokens[rng.random(B) < 0.02] = -3
        lacked += int((both.step(tokens) > 0).sum())
    assert B < 3 or lacked > 0
    both.step(np.zeros(B))
    assert both.nf == pages


def test_reserve_extremes(S):
    """Lengths near 2^31, nothing free, nothing held, no pages, no table."""
    import torch

    both = Both(S, np.random.default_rng(0), 4, 3, 64, 5)
    both.step([2 ** 31 - 1, -2 ** 31, 192, 1])   # the first can never fit and keeps nobody waiting
    both.step([64, 64, 192, 1])                  # one page left: the second waits
    both.step([64, 64, 0, 1])
    none = S.PagePool(0, 64)
    table, held = i32(np.zeros((2, 0))).view(2, 0), i32([0, 0])
    assert none.reserve(table, held, i32([0, 65])).tolist() == [0, 2]
    assert none.reserve(i32(np.full((1, 4), -1)), i32([0]), i32([65])).tolist() == [2]
    pool = S.PagePool(8, 64)
    assert pool.free.tolist() == list(range(8)) and int(pool.num_free) == 8
    # counts that cannot be are clamped, and nothing is written outside
    pool.num_free.fill_(100)
    table, held = i32(np.full((2, 4), -1)), i32([-5, 99])
    guard = torch.full((64,), 7, dtype=torch.int32, device="cuda")
    missing = pool.reserve(table, held, i32([256, 0]))
    assert missing.tolist() == [0, 0] and held.tolist() == [4, 0]
    assert int(pool.num_free) == 8 and guard.eq(7).all()
    assert pool.reserve(i32(np.zeros((0, 4))), i32([]), i32([])).numel() == 0


@pytest.mark.parametrize("B,width,page,N", [
    (1, 1, 32, 1), (1, 4, 64, 200), (5, 9, 96, 700), (64, 8, 64, 1088), (64, 8, 64, 1000),
    (256, 20, 32, 20000), (1024, 3, 64, 3000), (1500, 3, 64, 4097), (5000, 2, 64, 9001),
    (3, 4, 17, 0)])
def test_layout(S, B, width, page, N):
    """More rows than tokens and fewer; empty requests, tokens past the table, unmapped pages."""
    rng = np.random.default_rng(B + N)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    table[rng.random(table.shape) < 0.05] = -1
    table[rng.random(table.shape) < 0.05] = B * width
    mean = max(1, N // B)
    count = rng.integers(0, 2 * mean, B)
    count[rng.random(B) < 0.2] = 0
    count[rng.random(B) < 0.02] = -4
    start = rng.integers(0, max(1, width * page - mean), B)
    start[rng.random(B) < 0.02] = -9
    pool = S.PagePool(B * width, page)
    got = pool.layout(i32(table), i32(start), i32(count), N)
    want = M.layout(table, start, count, N, page, B * width)
    for name, g, w in zip(got._fields, got, want):
        assert np.array_equal(g.cpu().numpy(), w), name


def test_layout_extremes(S):
    """Positions up to the last, counts past everything, slots past 2^31, rows of nobody."""
    pool = S.PagePool(2 ** 31 - 1, 2048)
    table = i32([[5, 2 ** 31 - 2]])
    got = pool.layout(table, i32([2040]), i32([2 ** 31 - 1]), 20)
    assert got.offsets.tolist() == [0, 20] and got.seq_lens.tolist() == [2060]
    assert got.slots.tolist() == [5 * 2048 + 2040 + i for i in range(8)] + \
        [(2 ** 31 - 2) * 2048 + i for i in range(12)]
    got = pool.layout(table, i32([2 ** 31 - 4]), i32([9]), 5)
    assert got.offsets.tolist() == [0, 3] and got.seq_lens.tolist() == [2 ** 31 - 1]
    assert got.position.tolist() == [2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2, -1, -1]
    assert got.slots.tolist() == [-1] * 5
    got = pool.layout(i32(np.zeros((0, 2))), i32([]), i32([]), 3)
    assert got.offsets.tolist() == [0] and got.request.tolist() == [-1] * 3
    many = i32(np.full(3000, 2 ** 31 - 1))
    got = pool.layout(i32(np.zeros((3000, 1))), i32(np.zeros(3000)), many, 2500)
    assert got.offsets.tolist() == [0] + [2500] * 3000


def test_streams_and_outputs(S):
    """On another stream, into the caller's outputs."""
    import torch

    st = torch.cuda.Stream()
    table, start, count = i32([[3, 1], [2, 0]]), i32([60, 0]), i32([10, 3])
    pool = S.PagePool(4, 64)
    want = pool.layout(table, start, count, 15)
    out = S.StepLayout(*[torch.zeros_like(t) for t in want])
    torch.cuda.synchronize()
    got = pool.layout(table, start, count, 15, stream=st)
    same = pool.layout(table, start, count, 15, out=out, stream=st)
    st.synchronize()
    assert same is out
    for a, b, c in zip(want, got, out):
        assert torch.equal(a, b) and torch.equal(a, c)
