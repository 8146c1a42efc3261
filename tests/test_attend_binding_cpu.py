"""CPU checks of attention's binding and statuses beside tests/test_attend_cpu.py."""

import pytest

import fp8_quant_gb300 as kv
from fp8_quant_gb300 import build as kvbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    kvbuild.build()
    return kv.load_library()


def test_status_of_a_wait():
    assert kv.kv_status_str(5) == "KV_ERR_WAIT" and kv.KVStatus(5).name == "ERR_WAIT"
