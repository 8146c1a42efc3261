"""Attention at the edges of what its layouts may be: far strides, pages that no row needs, bytes next to a row's own."""

import pytest

torch = pytest.importorskip("torch")

from attncheck import AttendProblem

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")
WIDE = 60000    # tokens that a table row has room for: short sequences then take the kernels of long ones


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def tensors(p, wide):
    d = p.tensors(torch.device("cuda"))
    if wide:
        t = d["table"]
        d["table"] = torch.full((t.shape[0], WIDE // p.page), -1, dtype=torch.int32, device="cuda")
        d["table"][:, :t.shape[1]] = t
    return d


SLOT = (1 << 28) + (1 << 26)    # 7 and 8 of them pass 2^31


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("wide,nq", [(False, 1), (False, 3), (True, 1), (False, 40)])
def test_slot_strides_beyond_28_bits(wide, nq, fmt):
    """A slot-major cache ([page_size, pages, H, D]): rows of one page lie 320 MB apart."""
    p = AttendProblem([90, 33, 17], [nq, 1, nq], 8, 4, 64, fmt=fmt, seed=51)
    d = tensors(p, wide)
    big = torch.empty(p.page * SLOT, dtype=torch.uint8, device="cuda")
    at = 0
    for n in ("kc", "vc"):
        t = d[n]
        eb, (pages, _, H, W) = t.element_size(), t.shape
        d[n] = big.view(t.dtype).as_strided(t.shape, (H * W, SLOT // eb, W, 1), at // eb)
        d[n].copy_(t)
        at += pages * H * W * eb
    assert at <= SLOT
    p.check(p.attend(d))
