"""Rules of the paged history cache's kernels that only their source shows."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "cvr_ranking_model_gb300", "csrc")


@pytest.mark.parametrize("name", ["k_kv_attn.cuh", "k_kv_pages.cu", "cvr_kv.cuh"])
def test_no_read_only_loads(name):
    """The kernels of a stream start while earlier ones of it still write (programmatic dependent launch): what they read is not
    read-only for their lifetime, which loads of the read-only path and restricted pointers ask for."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict", code)
