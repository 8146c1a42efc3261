"""The cache of latent rows at the ends of the number range, and what a query makes of an infinite row that it sees."""

import numpy as np
import pytest

from attncheck import E4M3_ALL, bits_to_f32, e4m3_codes
from latentcheck import LatentProblem, StoreProblem, to_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def bf16_bits(x):
    """Of values that bf16 holds exactly."""
    bits = np.asarray(x, np.float32).view(np.uint32)
    assert (bits & 0xFFFF == 0).all()
    return (bits >> 16).astype(np.uint16)


# The largest magnitudes of rows: bf16's smallest number, its smallest normal one, around 448 / (the largest fp32), where the
# factor 448 / m would leave fp32's range, and ordinary ones.
TOPS = [2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -123, 2.0 ** -120, 2.0 ** -119, 2.0 ** -118, 2.0 ** -64, 1.0]


def tiny(L, norm=False):
    """A row for each of TOPS: its largest, halves and eighths of it, and zeros between them; rotary dims all zero."""
    T = len(TOPS)
    p = StoreProblem(T, L, 64, fmt="e4m3fn", norm=norm, seed=61)
    p.r[:] = 0
    shape = np.zeros(L, np.float32)
    shape[0:L:4], shape[1:L:4], shape[2:L:8] = 1.0, -0.5, 0.125
    x = shape[None] * np.array(TOPS, np.float64)[:, None]
    keep = np.abs(x) >= 2.0 ** -133         # what bf16 holds
    p.c = bf16_bits(np.where(keep, x, 0.0).astype(np.float32))
    return p


@pytest.mark.parametrize("L", [256, 512, 33])
def test_codes_of_rows_of_tiny_values(L):
    """Rows whose factor 448 / m is beyond fp32: the codes are those of the same row 2^64 times as large."""
    import fp8_quant_gb300 as kv
    p = tiny(L)
    d = p.tensors("cuda")
    p.call(d)
    at = torch.from_numpy(p.slots).cuda()
    codes = d["cache"].reshape(-1, L + 64)[at].cpu().numpy()
    scales = d["scales"][at, 0].cpu().numpy()
    c = bits_to_f32(p.c, "bf16")
    top = np.abs(c).max(1)
    assert np.array_equal(top.astype(np.float64), TOPS)
    # every value a power of two: the factor and the products in fp32, with the range that rows 2^64 times as large have
    up = np.where(top < 1e-19, np.float32(2.0 ** 64), np.float32(1.0)).astype(np.float32)
    factor = np.float32(448.0) / (top * up)
    want = e4m3_codes(((c * up[:, None]) * factor[:, None]).astype(np.float32))
    assert np.array_equal(codes[:, :L], want)
    assert (codes[:, L:] & 0x7F == 0).all()
    assert np.array_equal(scales, (top / np.float32(448.0)).astype(np.float32))
    # the values back: a code is off by half a step, the scale by half of fp32's smallest number
    got = E4M3_ALL[codes[:, :L]] * scales[:, None].astype(np.float64)
    assert (np.abs(got - c) <= 2.0 ** -4 * np.abs(c) + 2.0 ** -10 * scales[:, None] * 1.001 + 448 * 2.0 ** -150).all()
    out = torch.empty((len(TOPS), L + 64), dtype=torch.bfloat16, device="cuda")
    kv.kv_gather_latent(d["cache"], out, at, page_size=p.page, fmt="e4m3fn", scales=d["scales"], err=d["err"])
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("L", [256, 33])
def test_codes_of_rows_that_a_weight_makes_tiny(L):
    """The same after a norm, whose weights are 2^-123 and 2^-126."""
    p = StoreProblem(9, L, 64, fmt="e4m3fn", norm=True, seed=62)
    p.r[:] = 0
    p.c[:, ::3] = 0
    p.w = bf16_bits(np.where(np.arange(L) % 2, 2.0 ** -123, 2.0 ** -126).astype(np.float32))
    d = p.tensors("cuda")
    p.call(d)
    at = torch.from_numpy(p.slots).cuda()
    codes = d["cache"].reshape(-1, L + 64)[at].cpu().numpy()
    scales = d["scales"][at, 0].cpu().numpy().astype(np.float64)
    want, off = p.rows()
    assert (codes[:, :L][:, ::3] & 0x7F == 0).all()
    got = E4M3_ALL[codes] * scales[:, None]
    # (rows() adds 2^-140 for the norm of ordinary rows; fp32's own smallest step is 2^-149)
    off = np.minimum(off, np.abs(want) * 2.0 ** -17) + 2.0 ** -148
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -12) + 2.0 ** -10 * scales[:, None] * (1 + 2.0 ** -12) + 2 * off +
            448 * 2.0 ** -149).all()


def test_attention_over_rows_of_tiny_values():
    """One such row among ordinary ones does not reach the outputs of the queries that see it."""
    import fp8_quant_gb300 as kv
    L = 256
    p = tiny(L)
    d = p.tensors("cuda")
    d["indices"] = torch.arange(len(TOPS), device="cuda")
    p.call(d)
    q = torch.randn(1, 8, L + 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(63)).to(torch.bfloat16)
    n = torch.tensor([len(TOPS)], dtype=torch.int32, device="cuda")
    out = kv.kv_attend_latent(q, d["cache"], torch.zeros((1, 1), dtype=torch.int32, device="cuda"), n, latent_dim=L, fmt="e4m3fn",
                              scales=d["scales"], err=d["err"])
    rows = E4M3_ALL[d["cache"][0, :len(TOPS), 0].cpu().numpy()] * d["scales"][:len(TOPS)].cpu().numpy().astype(np.float64)
    x = bits_to_f32(to_bits(q), "bf16").astype(np.float64)[0]
    w = np.exp(x @ rows.T / np.sqrt(L + 64))
    want = (w / w.sum(-1, keepdims=True)) @ rows[:, :L]
    got = out.double().cpu().numpy()[0]
    assert np.isfinite(want).all() and np.isfinite(got).all()
    # the output's rounding, the weights', and the scores' (fp32 sums of 320 products, queries at 2^-25 of their largest)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * np.abs(rows).max()).all()


@pytest.mark.parametrize("fmt,what", [(None, np.inf), (None, -np.inf), ("e4m3fn", np.inf)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("batch", [([90, 4, 333, 64], [4, 4, 2, 3]), ([300, 129, 1000], [65, 128, 311]), ([1, 40, 700], [1, 1, 1])])
def test_what_an_infinite_row_gives(batch, dtype, fmt, what):
    """An infinite value (or scale) at each sequence's last key. Its last query has a score of infinity, and is NaN throughout, or of
    minus infinity, and then a weight of 0, which times the infinite value is NaN in that dim and nothing in the others; earlier
    queries do not see it."""
    lens, nqs = batch
    p = LatentProblem(lens, nqs, 4, 256, 64, dtype=dtype, fmt=fmt, seed=64)
    for b, n in enumerate(lens):
        at = p.table[b, (n - 1) // p.page], (n - 1) % p.page
        if fmt is None:
            p.cache[at][3] = ((0x7F80 if dtype == "bf16" else 0x7C00) | (0x8000 if what < 0 else 0))
            p.value[at][3] = what
        else:
            p.scales[at] = what
            with np.errstate(invalid="ignore"):
                p.value[at] = E4M3_ALL[p.cache[at]] * what
    d = p.tensors("cuda")
    lse = torch.zeros((sum(nqs), 4), device="cuda")
    out = p.attend(d, lse=lse)
    got = out.float().cpu().numpy()
    last = p.q_start[1:] - 1
    rest = np.setdiff1d(np.arange(sum(nqs)), last)
    assert np.isfinite(got[rest]).all()
    if fmt is None:
        assert np.isnan(got[last][..., 3]).all()
        q3 = bits_to_f32(p.q, dtype)[last][..., 3] * what
        alone = np.array(lens) == 1      # nothing but a score of -infinity: 0 / 0
        whole = (q3 > 0) | alone[:, None]
        assert np.isnan(got[last])[whole].all()
        assert (np.isnan(got[last])[~whole].sum(-1) == 1).all()
    else:
        assert np.isnan(got[last]).all()
    if 1 not in lens:
        p.check(out, lse)
