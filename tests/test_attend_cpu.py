"""CPU checks of the rotated append, the 4-bit gather and attention: host-side argument
validation (nothing is launched), the binding's checks, the strides it passes on, and the 64-bit
helpers against independent values."""

import numpy as np
import pytest
import torch

import fp8_quant_gb300 as kv
import oracle
from attncheck import (E4M3, AttendProblem, e2m1_codes, e4m3_codes, fp4_rows, fp4_values, rope_table,
                       rotated)
from fp8_quant_gb300 import build as kvbuild

A = 0x10000                                     # a device address nothing reads
INVALID, UNSUPPORTED, CUDA = (kv.KVStatus.ERR_INVALID_ARG, kv.KVStatus.ERR_UNSUPPORTED, kv.KVStatus.ERR_CUDA)
S = (4096, 256, 2, 4096, 256, 2, 2048, 256, 2, 2048, 256, 2)
S8 = S[:6] + (1024, 128, 1, 1024, 128, 1)
S4 = S[:6] + (512, 64, 1, 512, 64, 1)
SC = (A, A, 1024, 64, 8, 1024, 64, 8)


@pytest.fixture(scope="module", autouse=True)
def lib():
    kvbuild.build()
    return kv.load_library()


def rope(**over):
    r = dict(cos_sin=A, cos_sin_stride=128, max_position=100, positions=A, position_dtype=0,
             position_stride=1, rotary_dim=128, interleaved=0, q=A, q_out=A, num_q_heads=32,
             q_token=8192, q_head=256, qo_token=8192, qo_head=256)
    a = dict(k=A, v=A, k_cache=A, v_cache=A, indices=A, index_dtype=0, index_stride=1, num_tokens=4,
             num_heads=8, head_dim=128, src_dtype=1, strides=S, page_size=16, kc_page_stride=32768,
             vc_page_stride=32768, size_limit=100, rope=r, fmt=0, inv_k_scale=None, inv_v_scale=None,
             scales=None, d_err=A, stream=None)
    for n, x in over.items():
        (r if n in r else a)[n] = x
    if a["rope"] is not None:
        a["rope"] = tuple(r.values())
    return kv.raw.kv_store_rope(**a)


@pytest.mark.parametrize("over", [
    dict(num_tokens=-1), dict(k=None), dict(v_cache=None), dict(indices=None), dict(d_err=None), dict(d_err=A + 4),
    dict(index_dtype=3), dict(index_stride=0), dict(num_heads=0), dict(head_dim=0), dict(src_dtype=2), dict(page_size=0),
    dict(size_limit=-1), dict(fmt=3), dict(fmt=-1), dict(rope=None), dict(cos_sin=None), dict(cos_sin=A + 2), dict(positions=None),
    dict(position_dtype=2), dict(position_stride=0), dict(max_position=-1), dict(rotary_dim=-2), dict(rotary_dim=127),
    dict(rotary_dim=130), dict(cos_sin_stride=100), dict(q_out=None), dict(num_q_heads=0), dict(indices=A + 2),
    dict(index_dtype=1, indices=A + 4), dict(positions=A + 1), dict(k=A + 1), dict(q=A + 1), dict(q_token=8191), dict(qo_head=255),
    dict(k_cache=A + 1), dict(kc_page_stride=32767), dict(fmt=1, strides=S8, inv_k_scale=A + 2),
    dict(fmt=2, strides=S4), dict(fmt=2, strides=S4, scales=(None,) + SC[1:])])
def test_kv_store_rope_rejects_bad_arguments(over):
    assert rope(**over) == INVALID


@pytest.mark.parametrize("over", [
    dict(fmt=2, strides=S4, scales=SC, head_dim=120, rotary_dim=64), dict(fmt=2, strides=S4[:8] + (2,) + S4[9:], scales=SC),
    dict(num_tokens=1 << 41)])
def test_kv_store_rope_unsupported(over):
    assert rope(**over) == UNSUPPORTED


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@no_gpu
@pytest.mark.parametrize("over", [
    dict(), dict(q=None, q_out=None, num_q_heads=0), dict(rotary_dim=0, cos_sin=None), dict(fmt=1, strides=S8, inv_k_scale=A),
    dict(fmt=2, strides=S4, scales=SC), dict(fmt=1, strides=S8, k_cache=A + 1)])
def test_valid_appends_need_a_gpu(over):
    assert rope(**over) == CUDA


def test_empty_batches_are_ok():
    assert rope(num_tokens=0, k=None, indices=None, d_err=None, rope=None) == 0
    assert gather(num_tokens=0, k_out=None) == 0
    assert attend(num_seqs=0, q=None) == 0 and attend(num_q_tokens=0, q=None) == 0


def gather(**over):
    a = dict(k_cache=A, v_cache=A, scales=SC, k_out=A, v_out=A, indices=A, index_dtype=1, index_stride=1, num_tokens=4,
             num_heads=8, head_dim=128, out_dtype=0, strides=S4, page_size=16, kc_page_stride=8192,
             vc_page_stride=8192, size_limit=100, k_scale=None, v_scale=None, d_err=A, stream=None)
    a.update(over)
    return kv.raw.kv_gather_fp4(**a)


@no_gpu
@pytest.mark.parametrize("over,want", [
    (dict(num_tokens=-1), INVALID), (dict(k_out=None), INVALID), (dict(scales=None), INVALID),
    (dict(scales=(A, None) + SC[2:]), INVALID), (dict(out_dtype=5), INVALID), (dict(page_size=0), INVALID),
    (dict(k_scale=A + 1), INVALID), (dict(indices=A + 4), INVALID), (dict(k_out=A + 1), INVALID),
    (dict(strides=(4095,) + S4[1:]), INVALID), (dict(head_dim=72), UNSUPPORTED),
    (dict(strides=S4[:2] + (4,) + S4[3:]), UNSUPPORTED), (dict(), CUDA)])
def test_kv_gather_fp4_arguments(over, want):
    assert gather(**over) == want


ST = (8192, 256, 8192, 256, 32768, 2048, 256, 32768, 2048, 256)


def attend(**over):
    a = dict(q=A, out=A, lse=None, k_cache=A, v_cache=A, page_table=A, table_stride=8, table_width=8, seq_lens=A,
             q_start=None, num_seqs=4, num_q_tokens=4, num_q_heads=32, num_heads=8, head_dim=128, dtype=1, strides=ST,
             page_size=16, num_pages=64, fmt=0, k_scale=None, v_scale=None, scales=None, sm_scale=0.1, window=0, sinks=0,
             work=None, work_bytes=0, d_err=A, stream=None)
    a.update(over)
    return kv.raw.kv_attend(**a)


@no_gpu
@pytest.mark.parametrize("over,want", [
    (dict(num_seqs=-1), INVALID), (dict(num_q_tokens=-1), INVALID), (dict(fmt=4), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(k_cache=None), INVALID), (dict(page_table=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(strides=None), INVALID), (dict(d_err=None), INVALID), (dict(dtype=2), INVALID), (dict(num_heads=0), INVALID),
    (dict(num_heads=5), INVALID), (dict(num_q_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(page_size=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(table_width=0), INVALID), (dict(table_stride=7), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(work_bytes=-1), INVALID), (dict(sm_scale=float("nan")), INVALID),
    (dict(sm_scale=float("inf")), INVALID), (dict(num_q_tokens=5), INVALID), (dict(page_table=A + 2), INVALID),
    (dict(lse=A + 1), INVALID), (dict(d_err=A + 4), INVALID), (dict(work=A + 128, work_bytes=512), INVALID),
    (dict(fmt=2), INVALID), (dict(fmt=2, scales=(A, None) + SC[2:]), INVALID), (dict(k_scale=A + 2), INVALID),
    (dict(q=A + 1), UNSUPPORTED), (dict(k_cache=A + 1), UNSUPPORTED), (dict(head_dim=1025), UNSUPPORTED),
    (dict(fmt=2, scales=SC, head_dim=72), UNSUPPORTED), (dict(num_q_tokens=1 << 31, q_start=A), UNSUPPORTED),
    (dict(), CUDA), (dict(q_start=A, num_q_tokens=9), CUDA), (dict(fmt=1, k_cache=A + 1), CUDA),
    (dict(work=A, work_bytes=1 << 20), CUDA)])
def test_kv_attend_arguments(over, want):
    assert attend(**over) == want


# -- the binding ---------------------------------------------------------------------------


@pytest.fixture
def calls(monkeypatch):
    got = []
    for name in ("kv_store_rope", "kv_gather_fp4", "kv_attend"):
        monkeypatch.setattr(kv.raw, name, lambda *a, name=name: got.append((name, a)) or 0)
    monkeypatch.setattr(kv, "_stream_handle", lambda stream, device: 1234)
    return got


def rows(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_of_the_append(calls):
    T, HQ, H, D, pages, ps = 3, 8, 2, 64, 4, 16
    qkv = rows(T, (HQ + 2 * H) * D)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((HQ * D, H * D, H * D), 1))
    kc = rows(pages, H, ps, D).transpose(1, 2)              # pages of [H, page_size, D]
    pos, slots, tab, err = torch.arange(T), torch.arange(2 * T, dtype=torch.int32)[::2], torch.zeros(9, 32), torch.zeros(2, dtype=torch.int64)
    out = kv.kv_store_rope(k, v, kc, kc, slots, pos, tab, q=q, page_size=ps, interleaved=True, err=err)
    (_, a), = calls
    assert out.shape == q.shape and out.is_contiguous()
    assert a[5:11] == (0, 2, T, H, D, 1)
    assert a[11] == (1536, 128, 2, 1536, 128, 2, 128, 2048, 2, 128, 2048, 2)
    assert a[12:16] == (ps, 4096, 4096, pages * ps)
    assert a[16][1:8] == (32, 9, pos.data_ptr(), 1, 1, 32, 1) and a[16][10:] == (HQ, 1536, 128, 1024, 128)
    assert a[17:21] == (0, None, None, None)
    c4, s4 = torch.zeros(64, H, D // 2, dtype=torch.uint8), torch.zeros(64, H, D // 16, dtype=torch.uint8)
    assert kv.kv_store_rope(k, v, c4, c4, slots, pos, tab, page_size=ps, fmt="e2m1", k_scales=s4, v_scales=s4, err=err) is None
    a = calls[-1][1]
    assert a[11][6:] == (64, 32, 1, 64, 32, 1) and a[13] == 16 * 64 and a[17] == 2
    assert a[20][2:] == [16 * 8, 8, 4] * 2


@pytest.mark.parametrize("change,error", [
    (dict(fmt="int4"), ValueError), (dict(fmt="e2m1"), TypeError), (dict(pos=torch.arange(2)), ValueError),
    (dict(pos=torch.arange(3).float()), TypeError), (dict(tab=torch.zeros(9, 64, dtype=torch.float64)), TypeError),
    (dict(kc=rows(64, 3, 64)), ValueError), (dict(kc=rows(64, 2, 32)), ValueError), (dict(kc=rows(64, 128)), ValueError),
    (dict(kc=torch.zeros(64, 2, 64, dtype=torch.float16)), TypeError), (dict(q=rows(2, 8, 64)), ValueError),
    (dict(q=rows(3, 64, 8).transpose(1, 2)), ValueError), (dict(q_out=rows(3, 8, 64)), ValueError),
    (dict(k=torch.zeros(3, 2, 64)), ValueError), (dict(k=torch.zeros(3, 2, 64), v=torch.zeros(3, 2, 64)), TypeError),
    (dict(inv_k_scale=torch.ones(1)), ValueError)])
def test_binding_of_the_append_refuses(calls, change, error):
    a = dict(k=rows(3, 2, 64), v=rows(3, 2, 64), kc=rows(64, 2, 64), pos=torch.arange(3), tab=torch.zeros(9, 64), q=None,
             q_out=None, fmt=None, inv_k_scale=None)
    a.update(change)
    with pytest.raises(error):
        kv.kv_store_rope(a["k"], a["v"], a["kc"], rows(64, 2, 64) if a["kc"].shape == (64, 2, 64) else a["kc"],
                         torch.arange(3), a["pos"], a["tab"], q=a["q"], q_out=a["q_out"], fmt=a["fmt"],
                         inv_k_scale=a["inv_k_scale"], err=torch.zeros(2, dtype=torch.int64))
    assert not calls


def test_binding_of_attention(calls):
    q, kc = rows(5, 8, 64), rows(4, 16, 2, 64)
    table, lens, err = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    work = torch.empty(4096, dtype=torch.uint8)
    start = torch.zeros(3, dtype=torch.int32)
    out = kv.kv_attend(q, kc, kc, table, lens, q_start=start, window=9, sinks=2, work=work, err=err)
    (_, a), = calls
    assert a[1] == out.data_ptr() and a[6:8] == (3, 3) and a[10:16] == (2, 5, 8, 2, 64, 1)
    assert a[16] == (1024, 128, 1024, 128, 4096, 256, 128, 4096, 256, 128)
    assert a[17:22] == (16, 4, 0, None, None) and a[22] is None and a[23] == 0.125 and a[24:26] == (9, 2)
    assert a[26:28] == (work.data_ptr(), 4096)


@pytest.mark.parametrize("change", [
    dict(q=rows(2, 7, 64)), dict(q=rows(2, 512)), dict(q=rows(3, 8, 64)), dict(kc=rows(64, 2, 64)), dict(kc=rows(4, 16, 2, 32)),
    dict(kc=torch.zeros(4, 16, 2, 64, dtype=torch.float16)), dict(table=torch.zeros(2, 3)), dict(table=torch.zeros(2, dtype=torch.int32)),
    dict(lens=torch.zeros(3, dtype=torch.int32)), dict(lens=torch.zeros(2)), dict(start=torch.zeros(2, dtype=torch.int32)),
    dict(out=rows(2, 8, 32)), dict(lse=torch.zeros(2, 7)), dict(fmt="e2m1"), dict(fmt="fp3"), dict(page_size=8)])
def test_binding_of_attention_refuses(calls, change):
    a = dict(q=rows(2, 8, 64), kc=rows(4, 16, 2, 64), table=torch.zeros(2, 3, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32), start=None, out=None, lse=None, fmt=None, page_size=None)
    a.update(change)
    with pytest.raises((ValueError, TypeError)):
        kv.kv_attend(a["q"], a["kc"], a["kc"], a["table"], a["lens"], q_start=a["start"], out=a["out"], lse=a["lse"],
                     fmt=a["fmt"], page_size=a["page_size"], work=torch.empty(256, dtype=torch.uint8),
                     err=torch.zeros(2, dtype=torch.int64))
    assert not calls


# -- the 64-bit helpers --------------------------------------------------------------------


def test_e4m3_codes_agree_with_the_oracle():
    x = np.concatenate((np.arange(1 << 16, dtype=np.uint32) << 16, [0x7F800000, 0xFF800000])).astype(np.uint32).view(np.float32)
    got = e4m3_codes(x)
    assert np.array_equal(got, oracle.e4m3fn_encode(x))


def test_e2m1_codes_by_search():
    """Against the nearest of all sixteen values, ties to the even code."""
    x = np.concatenate((np.linspace(-7, 7, 2801), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.0, -0.0]))
    vals = [0, .5, 1, 1.5, 2, 3, 4, 6]
    for a, c in zip(x, e2m1_codes(x)):
        d = [abs(abs(a) - v) for v in vals]
        best = [i for i in range(8) if d[i] == min(d)]
        assert (c & 7) == (best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0))
        assert (c >> 3) == int(np.signbit(a))
    assert list(e2m1_codes([np.nan, np.inf, -np.inf])) == [7, 7, 15]


def test_fp4_rows_keep_their_bounds():
    """A block's largest magnitude is met within the scale's rounding, every other within half a
    step of the codes at the block's scale."""
    x = np.random.default_rng(3).standard_normal((50, 64)).astype(np.float32)
    c, s = fp4_rows(x)
    v = fp4_values(c, s)
    amax = np.abs(x).reshape(50, 4, 16).max(-1)
    assert (np.abs(E4M3[s] * 6 / amax - 1) <= 2.0 ** -4 + 1e-6).all()
    assert (np.abs(v - x).reshape(50, 4, 16) <= (E4M3[s][..., None] * 1.0 + amax[..., None] * 2.0 ** -4)).all()
    assert not fp4_rows(np.zeros((1, 16), np.float32))[0].any()


def test_rotation_is_a_rotation():
    x = np.random.default_rng(4).standard_normal((7, 2, 8)).astype(np.float32)
    tab = rope_table(50, 8)
    for il in (False, True):
        y = rotated(x, tab, np.arange(7) * 7, il)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
        assert np.array_equal(rotated(x, tab, np.zeros(7, int), il), x)


def test_attention_reference_by_hand():
    """One head, one dim at a time: the reference against a loop over keys."""
    import math
    p = AttendProblem([9, 3], [4, 5], 2, 1, 2, window=3, sinks=1, page=4, seed=5)
    out, _, lse, _ = p.reference()
    from attncheck import bits_to_f32
    q = bits_to_f32(p.q, "bf16").astype(float)
    for b, (n, nq) in enumerate(zip(p.lens, p.nqs)):
        for i in range(nq):
            pos, row = n - nq + i, p.q_start[b] + i
            for h in range(2):
                num, den = np.zeros(2), 0.0
                for j in range(n):
                    if j <= pos and (j > pos - 3 or j < 1):
                        at = p.table[b, j // 4], j % 4, 0
                        w = math.exp(float(q[row, h] @ p.value[0][at]) / math.sqrt(2))
                        num, den = num + w * p.value[1][at], den + w
                if den == 0:
                    assert (out[row, h] == 0).all() and lse[row, h] == -np.inf
                else:
                    assert np.allclose(out[row, h], num / den) and np.isclose(lse[row, h], math.log(den))
