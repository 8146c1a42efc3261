"""What the CUDA sources may not hold: read as text, nothing is built or run."""

import os
import re

import pytest

from fp8_quant_gb300 import build as kvbuild

FILES = sorted(f for f in os.listdir(kvbuild.CSRC) if f.endswith((".cu", ".cuh", ".h")))


def code_of(name):
    """The file without its comments."""
    with open(os.path.join(kvbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_multicast_and_no_clusters(name):
    """One library serves calls on one GPU and ranks on several: no load, commit or store goes to another CTA's memory."""
    code = code_of(name)
    for word in ("multicast", "multimem", "ClusterDimension", "barrier.cluster", "mapa"):
        assert word not in code, word
