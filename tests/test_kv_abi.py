"""Refusals of cvr_kv_create that need no GPU, and null handles."""
import ctypes

import pytest

GOOD = dict(q_heads=8, kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_req=4, max_pages=8, k=1 << 20, v=1 << 21)


@pytest.fixture(scope="module")
def lib():
    import cvr_ranking_model_gb300 as cvr
    return cvr.lib()


def create(lib, **change):
    import cvr_ranking_model_gb300 as cvr
    h = ctypes.c_void_p()
    raw = {k: change.pop(k) for k in ("reserved",) if k in change}
    cfg = cvr.make_kv_config(**{**GOOD, **change})
    for k, x in raw.items():
        setattr(cfg, k, x)
    st = lib.cvr_kv_create(ctypes.byref(cfg), None, ctypes.byref(h))
    return st, h


@pytest.mark.parametrize("change", [
    dict(kv_heads=0), dict(kv_heads=257, q_heads=257), dict(q_heads=0), dict(q_heads=7), dict(q_heads=130), dict(head_dim=96), dict(head_dim=0),
    dict(head_dim=256), dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=512), dict(max_req=0), dict(max_req=65536),
    dict(max_pages=0), dict(max_pages=2 ** 27), dict(n_pages=0), dict(n_pages=2 ** 31), dict(dtype=2), dict(dtype=3), dict(dtype=0, cache_dtype=1),
    dict(cache_dtype=3), dict(window=-1), dict(reserved=1), dict(k=0), dict(k=(1 << 20) + 8), dict(v=(1 << 21) + 2), dict(v=1 << 20),
    dict(k_scale=1 << 22), dict(v_scale=1 << 22), dict(cache_dtype=2), dict(cache_dtype=2, k_scale=1 << 22),
    dict(cache_dtype=2, k_scale=1 << 22, v_scale=1 << 22), dict(cache_dtype=2, k_scale=(1 << 22) + 4, v_scale=1 << 23),
    # strides: negative, zero, not of 16 bytes, too large, overlapping rows
    dict(k_strides=(-2048, 1024, 64)), dict(k_strides=(2048, 0, 64)), dict(k_strides=(2048, 1024, 68)), dict(v_strides=(2 ** 40, 1024, 64)),
    dict(k_strides=(2048, 1024, 56)), dict(v_strides=(2040, 1024, 64)), dict(k_strides=(2048, 64, 64)), dict(k_strides=(64, 64 * 10, 64 * 10)),
    dict(cache_dtype=2, k_scale=1 << 22, v_scale=1 << 23, k_strides=(2048, 1024, 72)), dict(v=0, v_scale=1 << 22, k=0)])
def test_create_refuses(lib, change):
    st, h = create(lib, **change)
    assert st == 1 and not h.value


def test_null_arguments(lib):
    import cvr_ranking_model_gb300 as cvr
    h = ctypes.c_void_p()
    assert lib.cvr_kv_create(None, None, ctypes.byref(h)) == 1
    assert lib.cvr_kv_create(ctypes.byref(cvr.make_kv_config(**GOOD)), None, None) == 1
    assert lib.cvr_kv_tables(None, 0, None, None, None, None, 0, None, None, None, None, None, 0) == 1
    assert lib.cvr_kv_append(None, 0, None, None, 0, None, 0) == 1
    assert lib.cvr_kv_attend(None, 0, None, 0, None, None, 1.0, None, 0, None) == 1
    assert lib.cvr_kv_sync(None) == 1
    assert lib.cvr_kv_last_error(None) == b"null handle"
    lib.cvr_kv_destroy(None)


def test_every_status_has_a_text(lib):
    import cvr_ranking_model_gb300 as cvr
    from cvr_ranking_model_gb300 import binding
    texts = {lib.cvr_status_string(s) for s in binding.STATUS}
    assert len(texts) == len(binding.STATUS) and lib.cvr_status_string(8) == b"free pages ran out"
    assert cvr.KvCache and ctypes.sizeof(binding.KvConfig) == 10 * 4 + 8 + 16 + 48 + 16
