"""Rotated appends whose query heads do not fill whole passes of a warp, so that one warp holds rows of Q, K
and V side by side, some written as they are and some quantised."""

import pytest

pytest.importorskip("torch")

from test_gpu_rope import run

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("HQ,H,D,R", [(14, 2, 64, 64), (14, 2, 64, 32), (3, 1, 128, 128), (7, 3, 128, 96), (5, 5, 128, 64),
                                      (9, 3, 96, 96), (1, 2, 32, 32), (25, 5, 64, 0), (3, 3, 256, 192)])
@pytest.mark.parametrize("T", [1, 700])
def test_rows_of_all_kinds_in_a_warp(T, HQ, H, D, R, interleaved, fmt):
    run(T, HQ, H, D, R, "bf16", fmt, interleaved=interleaved, seed=9)
