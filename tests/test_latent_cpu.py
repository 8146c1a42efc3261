"""CPU checks of the cache of latent rows: host-side argument validation (nothing is launched), the binding's checks and
the strides it passes on."""

import pytest

import fp8_quant_gb300 as kv
from fp8_quant_gb300 import build as kvbuild

torch = pytest.importorskip("torch")

A = 0x10000                                     # a device address nothing reads
INVALID, UNSUPPORTED, CUDA = (kv.KVStatus.ERR_INVALID_ARG, kv.KVStatus.ERR_UNSUPPORTED, kv.KVStatus.ERR_CUDA)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@pytest.fixture(scope="module", autouse=True)
def lib():
    kvbuild.build()
    return kv.load_library()


def store(**over):
    r = dict(cos_sin=A, cos_sin_stride=64, max_position=100, positions=A, position_dtype=0, position_stride=1, rotary_dim=64,
             interleaved=0, q=A, q_out=A, num_q_heads=32, q_token=4096, q_head=128, qo_token=36864, qo_head=1152)
    st = dict(c_token=1152, r_token=1152, cache_page=18432, cache_slot=1152, scale_slot=1)
    a = dict(c=A, r=A, cache=A, indices=A, index_dtype=0, index_stride=1, num_tokens=4, latent_dim=512, rope_dim=64, src_dtype=1,
             strides=st, page_size=16, size_limit=100, weight=A, eps=1e-6, rope=r, fmt=0, scales=None, d_err=A, stream=None)
    for n, x in over.items():
        (r if n in r else st if n in st else a)[n] = x
    for n, x in (("rope", r), ("strides", st)):
        if a[n] is not None:
            a[n] = tuple(x.values())
    return kv.raw.kv_store_latent(**a)


@pytest.mark.parametrize("over", [
    dict(num_tokens=-1), dict(c=None), dict(r=None), dict(cache=None), dict(indices=None), dict(d_err=None), dict(d_err=A + 4),
    dict(strides=None), dict(rope=None), dict(index_dtype=3), dict(index_stride=0), dict(latent_dim=0), dict(rope_dim=-1),
    dict(src_dtype=2), dict(page_size=0), dict(size_limit=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(fmt=2), dict(fmt=-1), dict(fmt=1), dict(fmt=1, scales=A + 2), dict(fmt=1, scales=A, scale_slot=0), dict(cos_sin=None),
    dict(cos_sin=A + 2), dict(positions=None), dict(position_dtype=2), dict(position_stride=0), dict(max_position=-1),
    dict(rotary_dim=-2), dict(rotary_dim=63), dict(rotary_dim=66), dict(cos_sin_stride=63), dict(q_out=None), dict(num_q_heads=0),
    dict(indices=A + 2), dict(index_dtype=1, indices=A + 4), dict(positions=A + 1), dict(c=A + 1), dict(r=A + 1), dict(q=A + 1),
    dict(weight=A + 1), dict(c_token=1151), dict(qo_head=127), dict(cache=A + 1), dict(cache_slot=1151), dict(cache_page=1)])
def test_store_rejects_bad_arguments(over):
    assert store(**over) == INVALID


@pytest.mark.parametrize("over", [dict(latent_dim=1000), dict(latent_dim=1025, rope_dim=0), dict(num_tokens=1 << 41),
                                  dict(latent_dim=2 ** 31 - 1), dict(rope_dim=2 ** 31 - 1)])
def test_store_unsupported(over):
    assert store(**over) == UNSUPPORTED


@no_gpu
@pytest.mark.parametrize("over", [dict(), dict(q=None, q_out=None, num_q_heads=0), dict(rope_dim=0, r=None, rope=None),
                                  dict(rotary_dim=0, cos_sin=None), dict(fmt=1, scales=A), dict(fmt=1, scales=A, cache=A + 1),
                                  dict(weight=None), dict(eps=0.0)])
def test_valid_appends_need_a_gpu(over):
    assert store(**over) == CUDA


def gather(**over):
    st = dict(c_token=1152, r_token=0, cache_page=18432, cache_slot=1152, scale_slot=1)
    a = dict(cache=A, scales=None, out=A, indices=A, index_dtype=1, index_stride=1, num_tokens=4, row_dim=576, out_dtype=0, strides=st,
             page_size=16, size_limit=100, fmt=0, d_err=A, stream=None)
    for n, x in over.items():
        (st if n in st else a)[n] = x
    if a["strides"] is not None:
        a["strides"] = tuple(st.values())
    return kv.raw.kv_gather_latent(**a)


@no_gpu
@pytest.mark.parametrize("over,want", [
    (dict(num_tokens=-1), INVALID), (dict(cache=None), INVALID), (dict(out=None), INVALID), (dict(indices=None), INVALID),
    (dict(strides=None), INVALID), (dict(d_err=None), INVALID), (dict(d_err=A + 2), INVALID), (dict(out_dtype=5), INVALID),
    (dict(page_size=0), INVALID), (dict(size_limit=-1), INVALID), (dict(row_dim=0), INVALID), (dict(fmt=2), INVALID),
    (dict(fmt=1), INVALID), (dict(fmt=1, scales=A + 1), INVALID), (dict(fmt=1, scales=A, scale_slot=0), INVALID),
    (dict(indices=A + 4), INVALID), (dict(index_dtype=7), INVALID), (dict(index_stride=0), INVALID), (dict(out=A + 1), INVALID),
    (dict(c_token=1151), INVALID), (dict(cache_slot=3), INVALID), (dict(row_dim=1025), UNSUPPORTED), (dict(), CUDA),
    (dict(fmt=1, scales=A, cache=A + 1), CUDA)])
def test_gather_arguments(over, want):
    assert gather(**over) == want


def attend(**over):
    st = dict(q_token=36864, q_head=1152, o_token=32768, o_head=1024, cache_page=18432, cache_slot=1152, scale_slot=1)
    a = dict(q=A, out=A, lse=None, cache=A, scales=None, page_table=A, table_stride=8, table_width=8, seq_lens=A, q_start=None,
             num_seqs=4, num_q_tokens=4, num_q_heads=32, row_dim=576, latent_dim=512, dtype=1, strides=st, page_size=16, num_pages=64,
             fmt=0, sm_scale=0.1, work=None, work_bytes=0, d_err=A, stream=None)
    for n, x in over.items():
        (st if n in st else a)[n] = x
    if a["strides"] is not None:
        a["strides"] = tuple(st.values())
    return kv.raw.kv_attend_latent(**a)


@no_gpu
@pytest.mark.parametrize("over,want", [
    (dict(num_seqs=-1), INVALID), (dict(num_q_tokens=-1), INVALID), (dict(fmt=2), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(cache=None), INVALID), (dict(page_table=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(strides=None), INVALID), (dict(d_err=None), INVALID), (dict(dtype=2), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(row_dim=0), INVALID), (dict(latent_dim=0), INVALID), (dict(latent_dim=577), INVALID), (dict(page_size=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(table_width=0), INVALID), (dict(table_stride=7), INVALID), (dict(work_bytes=-1), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(sm_scale=float("inf")), INVALID), (dict(num_q_tokens=5), INVALID),
    (dict(page_table=A + 2), INVALID), (dict(seq_lens=A + 1), INVALID), (dict(lse=A + 2), INVALID), (dict(d_err=A + 4), INVALID),
    (dict(work=A + 16, work_bytes=4096), INVALID), (dict(fmt=1), INVALID), (dict(fmt=1, scales=A + 2), INVALID),
    (dict(fmt=1, scales=A, scale_slot=0), INVALID), (dict(row_dim=1025), UNSUPPORTED), (dict(q=A + 1), UNSUPPORTED),
    (dict(cache_slot=1151), UNSUPPORTED), (dict(o_head=3), UNSUPPORTED), (dict(page_size=2 ** 31), UNSUPPORTED),
    (dict(num_pages=2 ** 31), UNSUPPORTED), (dict(num_seqs=1 << 26, num_q_tokens=1 << 26, num_q_heads=64), UNSUPPORTED),
    (dict(), CUDA), (dict(lse=A, q_start=A, num_q_tokens=9), CUDA), (dict(work=A, work_bytes=1 << 20), CUDA),
    (dict(fmt=1, scales=A, cache=A + 1), CUDA), (dict(row_dim=7, latent_dim=3), CUDA)])
def test_attend_arguments(over, want):
    assert attend(**over) == want


def test_empty_batches_are_ok():
    assert store(num_tokens=0, c=None, indices=None, d_err=None, rope=None) == 0
    assert gather(num_tokens=0, out=None) == 0
    assert attend(num_seqs=0, q=None) == 0 and attend(num_q_tokens=0, q=None) == 0


# -- the binding ------------------------------------------------------------------------------------------------------

BF = torch.bfloat16


@pytest.fixture
def called(monkeypatch):
    got = {}
    for n in ("kv_store_latent", "kv_gather_latent", "kv_attend_latent"):
        monkeypatch.setattr(kv.raw, n, lambda *a, n=n: got.update({n: a}) or 0)
    monkeypatch.setattr(kv, "_stream_handle", lambda stream, device: 0)
    return got


def store_args(**over):
    a = dict(c=torch.zeros(3, 512, dtype=BF), r=torch.zeros(3, 64, dtype=BF), cache=torch.zeros(8, 16, 1, 576, dtype=BF),
             indices=torch.arange(3), positions=torch.arange(3), cos_sin=torch.zeros(9, 64), page_size=16, err=torch.zeros(2, dtype=torch.int64))
    a.update(over)
    return a


@pytest.mark.parametrize("over", [
    dict(c=torch.zeros(3, 512)), dict(c=torch.zeros(3, 1024, dtype=BF)[:, ::2]), dict(r=torch.zeros(3, 64, dtype=torch.float16)),
    dict(r=torch.zeros(2, 64, dtype=BF)), dict(r=None), dict(positions=None), dict(cos_sin=None), dict(cos_sin=torch.zeros(9, 64).double()),
    dict(positions=torch.arange(4)), dict(indices=torch.arange(2)), dict(indices=torch.arange(3).float()),
    dict(cache=torch.zeros(8, 16, 1, 512, dtype=BF)), dict(cache=torch.zeros(8, 16, 2, 576, dtype=BF)),
    dict(cache=torch.zeros(8, 16, 576, dtype=BF)), dict(cache=torch.zeros(8, 16, 1, 1152, dtype=BF)[..., ::2]),
    dict(cache=torch.zeros(8, 16, 1, 576, dtype=torch.float16)), dict(page_size=8), dict(page_size=0), dict(fmt="e2m1"),
    dict(fmt="e4m3fn"), dict(scales=torch.zeros(128, 1)), dict(weight=torch.zeros(512)), dict(weight=torch.zeros(64, dtype=BF)),
    dict(q=torch.zeros(3, 4, 32, dtype=BF)), dict(q=torch.zeros(2, 4, 64, dtype=BF)), dict(q_out=torch.zeros(3, 4, 64, dtype=BF)),
    dict(q=torch.zeros(3, 4, 64, dtype=BF), q_out=torch.zeros(3, 5, 64, dtype=BF)),
    dict(fmt="e4m3fn", cache=torch.zeros(8, 16, 1, 576, dtype=torch.uint8), scales=torch.zeros(64, 1)),
    dict(fmt="e4m3fn", cache=torch.zeros(8, 16, 1, 576, dtype=torch.uint8), scales=torch.zeros(128, 1).double())])
def test_store_binding_refuses(called, over):
    with pytest.raises((TypeError, ValueError)):
        kv.kv_store_latent(**store_args(**over))
    assert not called


def test_store_binding_passes_strides(called):
    both = torch.zeros(3, 640, dtype=BF)
    q, whole = torch.zeros(3, 4, 64, dtype=BF), torch.zeros(3, 4, 576, dtype=BF)
    cache = torch.zeros(8, 16, 1, 640, dtype=torch.uint8)[..., :576]
    out = kv.kv_store_latent(**store_args(c=both[:, :512], r=both[:, 512:576], q=q, q_out=whole[..., 512:], cache=cache, fmt="e4m3fn",
                                          scales=torch.zeros(128, 2)[:, :1], interleaved=True))
    a = called["kv_store_latent"]
    assert out.data_ptr() == whole.data_ptr() + 1024
    assert a[10] == (1280, 1280, 16 * 640, 640, 2) and a[6:9] == (3, 512, 64) and a[12] == 128 and a[16] == 1
    assert a[15][6:8] == (64, 1) and a[15][10:] == (4, 512, 128, 4608, 1152)


def test_store_binding_without_rotary_dims(called):
    kv.kv_store_latent(torch.zeros(3, 576, dtype=BF), None, torch.zeros(128, 1, 576, dtype=BF), torch.arange(3),
                       err=torch.zeros(2, dtype=torch.int64))
    a = called["kv_store_latent"]
    assert a[1] is None and a[15] is None and a[10][2:] == (1152, 1152, 1)
    with pytest.raises(ValueError):
        kv.kv_store_latent(torch.zeros(3, 576, dtype=BF), None, torch.zeros(128, 1, 576, dtype=BF), torch.arange(3), torch.arange(3))


@pytest.mark.parametrize("over", [
    dict(out=torch.zeros(3, 512, dtype=BF)), dict(out=torch.zeros(2, 576, dtype=BF)), dict(out=torch.zeros(3, 576)),
    dict(out=torch.zeros(3, 1152, dtype=BF)[:, ::2]), dict(indices=torch.zeros(3, 1, dtype=torch.int64)), dict(fmt="e5m2"),
    dict(fmt="e4m3fn"), dict(scales=torch.zeros(128))])
def test_gather_binding_refuses(called, over):
    a = dict(cache=torch.zeros(8, 16, 1, 576, dtype=BF), out=torch.zeros(3, 576, dtype=BF), indices=torch.arange(3), page_size=16,
             err=torch.zeros(2, dtype=torch.int64))
    a.update(over)
    with pytest.raises((TypeError, ValueError)):
        kv.kv_gather_latent(**a)
    assert not called


def attend_args(**over):
    a = dict(q=torch.zeros(2, 8, 576, dtype=BF), cache=torch.zeros(4, 16, 1, 576, dtype=BF), page_table=torch.zeros(2, 3, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), latent_dim=512, work=torch.zeros(4096, dtype=torch.uint8),
             err=torch.zeros(2, dtype=torch.int64))
    a.update(over)
    return a


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(2, 8, 512, dtype=BF)), dict(q=torch.zeros(2, 8, 1152, dtype=BF)[..., ::2]), dict(q=torch.zeros(2, 8, 576)),
    dict(q=torch.zeros(3, 8, 576, dtype=BF)), dict(latent_dim=0), dict(latent_dim=577), dict(cache=torch.zeros(64, 1, 576, dtype=BF)),
    dict(cache=torch.zeros(4, 16, 2, 576, dtype=BF)), dict(page_table=torch.zeros(2, 3)), dict(page_table=torch.zeros(3, 2, dtype=torch.int32).T),
    dict(seq_lens=torch.zeros(3, dtype=torch.int32)), dict(seq_lens=torch.zeros(2)), dict(q_start=torch.zeros(2, dtype=torch.int32)),
    dict(out=torch.zeros(2, 8, 576, dtype=BF)), dict(out=torch.zeros(2, 8, 512)), dict(lse=torch.zeros(2, 8).double()),
    dict(work=torch.zeros(4096, dtype=torch.uint8)[::2]), dict(fmt="e4m3fn"), dict(page_size=0), dict(page_size=8),
    dict(fmt="e4m3fn", cache=torch.zeros(4, 16, 1, 576, dtype=torch.uint8), scales=torch.zeros(63))])
def test_attend_binding_refuses(called, over):
    with pytest.raises((TypeError, ValueError)):
        kv.kv_attend_latent(**attend_args(**over))
    assert not called


def test_attend_binding_passes_strides(called):
    out = kv.kv_attend_latent(**attend_args(cache=torch.zeros(70, 1, 576, dtype=BF), page_size=16,
                                            q=torch.zeros(2, 8, 640, dtype=BF)[..., :576]))
    a = called["kv_attend_latent"]
    assert out.shape == (2, 8, 512) and a[16] == (10240, 1280, 8192, 1024, 16 * 1152, 1152, 1) and a[17:20] == (16, 4, 0)
    assert abs(a[20] - 1 / 24) < 1e-9
