"""Small weights beside a strong key: many that are far below the largest one's last bit in fp16 still add up."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attncheck import UNIT, AttendProblem, bits_to_f32, e4m3_codes, fp4_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def strong_first_key(lens, nqs, D, fmt, dtype, size):
    """Positive queries; key 0 of a sequence is `size` in every dim and has a value of 0; the others' values are positive."""
    import workloads as wl
    p = AttendProblem(lens, nqs, 2, 2, D, dtype=dtype, fmt=fmt, page=16, seed=71, scale=0.25)
    p.q &= 0x7FFF
    k, v = p.cache
    if fmt is None:
        v &= 0x7FFF
        key, val = wl.to_bits(np.float32([size]), dtype)[0], 0
    elif fmt == "e4m3fn":
        v &= 0x7F
        key, val = e4m3_codes(np.float32([size]) / p.kv_scale[0])[0], 0
    else:
        v &= 0x77
        key, val = 0x77, 0
    for b, n in enumerate(lens):
        at = p.table[b, 0], 0
        k[at], v[at] = key, val
        if fmt == "e2m1":
            p.scales[0][at] = e4m3_codes(np.float32([size]) / p.kv_scale[0] / np.float32(6.0))[0]
    if fmt is None:
        p.value = [bits_to_f32(c, dtype).astype(np.float64) for c in p.cache]
    elif fmt == "e4m3fn":
        from attncheck import E4M3_ALL
        p.value = [E4M3_ALL[c] * float(s) for c, s in zip(p.cache, p.kv_scale)]
    else:
        p.value = [fp4_values(c, s) * float(g) for c, s, g in zip(p.cache, p.scales, p.kv_scale)]
    return p


@pytest.mark.parametrize("fmt,dtype", [(None, "f16"), (None, "bf16"), ("e4m3fn", "bf16"), ("e2m1", "bf16"), ("e2m1", "f16")])
@pytest.mark.parametrize("size", [3.0, 6.2, 8.0])
@pytest.mark.parametrize("nq,wide", [(1, False), (3, True), (60, False)])
def test_small_weights_add_up(nq, wide, size, fmt, dtype):
    """As AttendProblem's bound, with fp16's last place 2^-24 under weights that begin at 2^7 or more: half a place
    of each of n weights, n 2^-32 max|v|, in place of n 2^-24 max|v|."""
    p = strong_first_key([3000, 700], [nq, 1], 64, fmt, dtype, size)
    d = p.tensors(torch.device("cuda"))
    if wide:
        t = d["table"]
        d["table"] = torch.full((2, 60000 // p.page), -1, dtype=torch.int32, device="cuda")
        d["table"][:, :t.shape[1]] = t
    out = p.attend(d).double().cpu().numpy()
    ref, bound, _, _ = p.reference()
    for b, n in enumerate(p.lens):
        j = np.arange(n)
        v = np.abs(p.value[1][p.table[b, j // p.page], j % p.page]).max((0, 2))     # of each head
        bound[p.q_start[b]:p.q_start[b + 1]] += n * v[:, None] * (2.0 ** -32 - 2.0 ** -24)
    assert (bound > 0).all() and UNIT[dtype] < 0.01
    worst = (np.abs(out - ref) / bound).max()
    assert worst <= 1.0, f"{worst:.3g} times the bound off"
