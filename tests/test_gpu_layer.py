"""The example layer: append with rotation, attention, and the captured decode step, run together."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attncheck as ac

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def cached(layer, table, n):
    """K and V of one sequence as the cache holds them: float64 [n, H, D]."""
    j = np.arange(n)
    at = table[j // layer.page_size], j % layer.page_size
    out = []
    for c, s, g in ((layer.k_cache, layer.k_scales, layer.forward_scale[0]),
                    (layer.v_cache, layer.v_scales, layer.forward_scale[1])):
        if layer.fmt is None:
            out.append(ac.bits_to_f32(bits(c)[at], "bf16").astype(np.float64))
            continue
        codes = c.cpu().numpy()[at]
        x = ac.E4M3_ALL[codes] if layer.fmt == "e4m3fn" else ac.fp4_values(codes, s.cpu().numpy()[at])
        out.append(x * float(g.item()))
    return out


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
@pytest.mark.parametrize("fmt", FMTS)
def test_last_step_against_the_cache(fmt, window, sinks):
    """The last step's outputs against 64 bits over the bytes in the cache. A bound as
    ac.AttendProblem's: |out' - out| <= u |out| + (u + 2 d) sum p |v| + n 2^-24 max|v|."""
    from fp8_quant_gb300.examples import attention_layer as ex
    layer, step, outs, rows = ex.generate((1, 77, 300, 1023), 4, fmt=fmt, window=window, sinks=sinks)
    table, q = step.table.cpu().numpy(), ac.bits_to_f32(bits(step.q_rot), "bf16").astype(np.float64)
    u, G, sm = ac.UNIT["bf16"], layer.HQ // layer.H, 1.0 / math.sqrt(layer.D)
    for b, r in enumerate(rows):
        n = r.shape[0]
        K, V = cached(layer, table[b], n)
        j = np.arange(n)
        see = (j > n - 1 - window) | (j < sinks) if window else j >= 0
        for h in range(layer.HQ):
            k, v, x = K[:, h // G], V[:, h // G], q[b, h]
            s = np.where(see, k @ x * sm, -np.inf)
            d = (np.abs(k) @ np.abs(x)).max() * sm * 2.0 ** -20 + \
                layer.D * 2.0 ** -25 * np.abs(x).max() * np.abs(k).max() * sm + 2.0 ** -20
            w = np.exp(s - s.max())
            w /= w.sum()
            o, a = w @ v, w @ np.abs(v)
            bound = u * np.abs(o) + (u + 2 * d) * a + n * 2.0 ** -24 * np.abs(v).max() + 2.0 ** -24
            assert (np.abs(outs[-1][b, h].double().cpu().numpy() - o) <= bound).all()


# root mean square of a value's relative error in each format: rounding to 8 bits of significand, to 4 bits
# (2^-4 at most), and to the 4-bit grid of a block of 16 (at most a sixth of the block's maximum, which
# for normal values is about 2.2 times their root mean square, less its zeros' part)
STEP = {None: 2.0 ** -8, "e4m3fn": 2.0 ** -4, "e2m1": 2.2 / 6}


@pytest.mark.parametrize("fmt", FMTS)
def test_near_the_unquantised_attention(fmt):
    """Quantised values leave the outputs' relative error below the values' own largest one: the error of a mean
    of n values with independent errors is no larger, relative to the mean, than one value's; the keys'
    errors shift the scores, whose size here is about 1, by at most as much, and the two add."""
    from fp8_quant_gb300.examples import attention_layer as ex
    layer, _, outs, rows = ex.generate((5, 200, 777), 3, fmt=fmt)
    want = torch.stack([ex.plain_attention(layer, r, layer.HQ) for r in rows])
    err = (outs[-1].double() - want).square().sum().sqrt() / want.square().sum().sqrt()
    assert err.item() <= 2 * STEP[fmt]


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_step_is_the_direct_one(fmt):
    """The same calls, replayed from a graph and made one by one: the same bits, and so in a second run."""
    from fp8_quant_gb300.examples import attention_layer as ex
    a, b, c = (ex.generate((3, 64, 65, 2000), 5, fmt=fmt, graph=g)[2] for g in (True, False, True))
    for x, y, z in zip(a, b, c):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(x.view(torch.int16), z.view(torch.int16))


def test_prefill_and_steps_agree():
    """A prompt taken at once and token by token writes the same cache bytes; the outputs differ by
    roundings only, at most two of the output's and two of the weights'."""
    from fp8_quant_gb300.examples import attention_layer as ex
    whole = ex.generate((40,), 1, seed=3)
    single = ex.generate((1,), 40, seed=3)
    assert torch.equal(whole[0].k_cache.view(torch.int16), single[0].k_cache.view(torch.int16))
    assert torch.equal(whole[0].v_cache.view(torch.int16), single[0].v_cache.view(torch.int16))
    v = whole[3][0][:, 40 * 128:].float().unflatten(1, (8, 128)).abs().amax().item()
    got = torch.cat([x for x in single[2]])[:40]
    assert (whole[2][0].float() - got.float()).abs().max().item() <= 4 * ac.UNIT["bf16"] * v


def test_admission_without_pages():
    from fp8_quant_gb300.examples import attention_layer as ex
    layer = ex.AttentionLayer(4, 1, 64, pages=3, page_size=16, max_position=64)
    layer.admit([30])
    with pytest.raises(RuntimeError, match="pages"):
        layer.admit([17])
