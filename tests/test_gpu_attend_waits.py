"""What a caller learns of a wait that ran out in an attention kernel, and that none does while a CTA is at work."""

import pytest

torch = pytest.importorskip("torch")

from attncheck import AttendProblem

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


@pytest.mark.parametrize("skipped", [0, 3])
def test_the_record_tells_a_wait_from_an_index(skipped):
    import fp8_quant_gb300 as kv
    err = kv.error_record()
    err[0] = skipped - 2 ** 63
    err[1] = ~5 if skipped else 0
    assert kv.kv_error_poll(err) == (kv.KVStatus.ERR_WAIT, skipped, 5 if skipped else -1)
    assert kv.kv_error_poll(err) == (kv.KVStatus.OK, 0, -1)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("long", [False, True])
def test_a_split_call_that_lost_a_part_gives_nan(long, fmt):
    """The mark that a CTA leaves in the workspace's head, set beforehand: no row is made of parts that may be missing."""
    import fp8_quant_gb300 as kv
    p = AttendProblem([3000, 70], [1, 2], 8, 2, 128, fmt=fmt, seed=61)
    d = p.tensors(torch.device("cuda"))
    if long:    # a table row long enough for the TMA-fed kernels
        t = d["table"]
        d["table"] = torch.full((2, 60000 // p.page), -1, dtype=torch.int32, device="cuda")
        d["table"][:, :t.shape[1]] = t
    work = torch.zeros(kv.ATTEND_WORK_BYTES, dtype=torch.uint8, device="cuda")
    lse = torch.zeros(3, 8, device="cuda")
    p.check(p.attend(d, work=work, lse=lse), lse)
    work.view(torch.int32)[1] = 1
    assert p.attend(d, work=work, lse=lse).isnan().all() and lse.isnan().all()
    work[:kv.ATTEND_HEAD_BYTES] = 0
    p.check(p.attend(d, work=work, lse=lse), lse)


def test_no_wait_runs_out_while_rows_are_done_again():
    """A NaN that every row sees has them done key by key, for seconds here: longer than any wait may last,
    and the CTA's next item waits all that time. (Which CTA has two items: as many blocks as SMs and more.)"""
    import numpy as np
    import fp8_quant_gb300 as kv
    lens = [64] * 200
    lens[120] = 200_000
    p = AttendProblem(lens, [40] * 200, 4, 1, 128, fmt="e4m3fn", page=64, seed=62)
    p.value[1][p.table[120, 0], 0] = np.nan
    p.cache[1][p.table[120, 0], 0] = 0x7F
    d = p.tensors(torch.device("cuda"))
    err = kv.error_record()
    out = torch.full_like(d["q"], 7.0)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    p.attend(d, out=out, err=err)
    end.record()
    assert kv.kv_error_poll(err) == (kv.KVStatus.OK, 0, -1)
    p.check(out)
    assert start.elapsed_time(end) > 2300      # it did take longer than a wait may


def test_a_wait_that_nothing_ends_runs_out(tmp_path):
    """The kernels' wait, on a barrier of its own: false for every warp, the record's bit beside its count, a live context."""
    import os
    import subprocess
    from fp8_quant_gb300 import build
    exe = str(tmp_path / "wait_limit")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "wait_limit.cu")
    subprocess.check_call([build.nvcc(), *build.NVCC_FLAGS, "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC, "-o", exe, src])
    got = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert got.returncode == 0 and got.stdout.split() == ["no", "error", "1", "0", "0", "1", "3"], got.stdout + got.stderr
