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


@pytest.mark.parametrize("wide,nq", [(False, 1), (True, 1), (True, 3), (False, 40)])
@pytest.mark.parametrize("D,H", [(32, 8), (96, 8), (96, 16), (80, 4), (112, 2), (48, 2), (160, 4)])
def test_block_scales_next_to_a_row(D, H, wide, nq):
    """NaN scales of another head or of a slot that no row sees leave every other row's bits as they are."""
    p = AttendProblem([333, 64, 50, 1], [nq, 1, nq, 1], 2 * H, H, D, fmt="e2m1", page=32, seed=52)
    d = tensors(p, wide)
    want = p.attend(d)
    p.check(want)
    used = torch.from_numpy(p.used).cuda()[..., None, None]
    clean = dict(d, ks=torch.where(used, d["ks"], 0), vs=torch.where(used, d["vs"], 0))
    assert torch.equal(p.attend(clean).view(torch.int16), want.view(torch.int16))
    dirty = dict(d, ks=d["ks"].clone(), vs=d["vs"].clone())
    for n in ("ks", "vs"):
        dirty[n][:, :, 1] = 0x7F
    got = p.attend(dirty)
    others = [h for h in range(2 * H) if h // 2 != 1]
    assert torch.equal(got[:, others].view(torch.int16), want[:, others].view(torch.int16))
    assert got[:, 2:4].isnan().all()
