"""Refusals of 4-bit configurations that need no GPU, null handles of the calls beside them, and rules that only the source shows."""
import ctypes
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "cvr_ranking_model_gb300", "csrc")
GOOD = dict(q_heads=8, kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_req=4, max_pages=8, k=1 << 20, v=1 << 21, cache_dtype=3, k_scale=1 << 22, v_scale=1 << 23)


@pytest.fixture(scope="module")
def lib():
    import cvr_ranking_model_gb300 as cvr
    return cvr.lib()


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(cache_dtype=4), dict(k_scale=0), dict(v_scale=0), dict(k_scale=0, v_scale=0), dict(v_scale=1 << 22), dict(k_scale=(1 << 22) + 8), dict(k=(1 << 20) + 8),
    dict(k=0), dict(head_dim=16), dict(head_dim=256),
    # strides in values, two to a byte: not of 16 bytes, overlapping rows, too large
    dict(k_strides=(2048, 1024, 80)), dict(k_strides=(2048, 1024, 48)), dict(v_strides=(2064, 1024, 64)), dict(k_strides=(2048, 64, 64)), dict(v_strides=(2 ** 41, 1024, 64)),
    dict(k_strides=(2048, 1024, 32))])
def test_create_refuses(lib, change):
    import cvr_ranking_model_gb300 as cvr
    h = ctypes.c_void_p()
    st = lib.cvr_kv_create(ctypes.byref(cvr.make_kv_config(**{**GOOD, **change})), None, ctypes.byref(h))
    assert st == 1 and not h.value


def test_null_handles(lib):
    assert lib.cvr_kv_read(None, 0, None, None, 0, None, 0) == 1
    assert lib.cvr_kv_weigh(None, 0, None, 0, None, None, None, 1.0, None, 1.0, None) == 1
    assert lib.cvr_kv_evict(None, 0, None, 2, 1, 0, 0, None, None, None, None, None, None, None, 0, None, None) == 1


def test_names():
    import cvr_ranking_model_gb300 as cvr
    assert cvr.DTYPE_FP4 == 3 and all(hasattr(cvr.KvCache, n) for n in ("read", "weigh", "evict"))
    with open(os.path.join(os.path.dirname(CSRC), os.pardir, "include", "cvr.h")) as f:
        assert "CVR_DTYPE_FP4 = 3" in f.read()


@pytest.mark.parametrize("name", ["cvr_kv_rows.cuh", "k_kv_weigh.cu", "k_kv_evict.cu", "k_kv_attn_fp4.cuh"])
def test_no_read_only_loads(name):
    """What a kernel reads may still be written when it starts (programmatic dependent launch)."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict", code)
