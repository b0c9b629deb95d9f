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
