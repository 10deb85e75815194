"""Refusals of the paged cache's entries that need no device, and checks of the plain forms
the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import paged_ref as ref
from quantized_attention_layer_gb300 import build, hfa


@pytest.fixture(scope="module")
def libhfa():
    build.build()
    return hfa.lib()


BASE = dict(num_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=10, max_pages=4, window=0, eps=1e-6,
            rope_theta=1e4, attn_scale=1.0, softcap=0.0, flags=0)


@pytest.mark.parametrize("change,status", [
    (dict(num_heads=7), "EINVAL"), (dict(num_kv_heads=0), "EINVAL"), (dict(num_heads=18), "EUNSUPPORTED"),
    (dict(head_dim=96), "EUNSUPPORTED"), (dict(head_dim=512), "EUNSUPPORTED"), (dict(page_size=8), "EUNSUPPORTED"),
    (dict(page_size=48), "EUNSUPPORTED"), (dict(num_pages=0), "EINVAL"), (dict(max_pages=0), "EINVAL"),
    (dict(num_pages=1 << 26), "EUNSUPPORTED"), (dict(max_pages=(1 << 20) + 1), "EINVAL"), (dict(window=-1), "EINVAL"),
    (dict(window=4, flags=hfa.HFA_F_BLOCK_BIDIR), "EINVAL"), (dict(flags=hfa.HFA_F_RING), "EINVAL"),
    (dict(eps=-1.0), "EINVAL"), (dict(eps=float("nan")), "EINVAL"), (dict(rope_theta=0.0), "EINVAL"),
    (dict(attn_scale=0.0), "EINVAL"), (dict(attn_scale=float("inf")), "EINVAL"), (dict(softcap=-1.0), "EINVAL")])
def test_create_refuses(libhfa, change, status):
    d = hfa.hfa_paged_desc(**{**BASE, **change})
    h = ctypes.c_void_p()
    st = libhfa.hfa_paged_create(ctypes.byref(d), None, None, None, None, ctypes.byref(h))
    assert st == getattr(hfa, "HFA_" + status), libhfa.hfa_paged_last_error(None)
    assert not h.value and libhfa.hfa_paged_last_error(None)


def test_create_refuses_factors_and_null(libhfa):
    d = hfa.hfa_paged_desc(**BASE)
    h = ctypes.c_void_p()
    f = np.ones(64, dtype=np.float32)
    for bad in (0.0, -1.0, np.inf, np.nan):
        f[5] = bad
        st = libhfa.hfa_paged_create(ctypes.byref(d), None, None, f.ctypes.data, None, ctypes.byref(h))
        assert st == hfa.HFA_EINVAL and b"factors[5]" in libhfa.hfa_paged_last_error(None)
    assert libhfa.hfa_paged_create(None, None, None, None, None, ctypes.byref(h)) == hfa.HFA_EINVAL
    assert libhfa.hfa_paged_create(ctypes.byref(d), None, None, None, None, None) == hfa.HFA_EINVAL


def test_null_handle(libhfa):
    assert libhfa.hfa_paged_destroy(None) == hfa.HFA_EINVAL
    assert libhfa.hfa_paged_check_status(None, None) == hfa.HFA_EINVAL
    assert libhfa.hfa_paged_workspace_bytes(None, 1, 1) == 0
    pages = hfa.hfa_pages()
    assert libhfa.hfa_paged_append(None, None, 1, None, None, None, None, None, 0, None, 0, None, 0, 0,
                                   ctypes.byref(pages), None) == hfa.HFA_EINVAL
    assert libhfa.hfa_paged_attention(None, None, 1, None, None, None, None, None, 0, 0, ctypes.byref(pages), None,
                                      0, None) == hfa.HFA_EINVAL
    assert libhfa.hfa_paged_read(None, None, 1, None, None, None, None, ctypes.byref(pages), 1, None,
                                 None) == hfa.HFA_EINVAL


def test_plain_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 64))
    y = ref.rotate_rows(x, [0, 1, 2, 100000, 7], 1e4, None)
    assert np.array_equal(y[0], x[0])
    assert np.allclose(ref.pair_len(y), ref.pair_len(x), rtol=1e-12)
    # scores depend on the distance alone
    a = ref.rotate_rows(x, [3] * 5, 1e4, None), ref.rotate_rows(x[::-1], [10] * 5, 1e4, None)
    b = ref.rotate_rows(x, [103] * 5, 1e4, None), ref.rotate_rows(x[::-1], [110] * 5, 1e4, None)
    assert np.allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1), rtol=1e-9)


def test_plain_append_and_attention_by_hand():
    # two slots of a page at scale 1, then a row whose maximum doubles the scale
    codes = np.zeros((1, 1, 16, 64), dtype=np.int8)
    codes[0, 0, :2] = 100
    rows = np.zeros((1, 1, 64))
    rows[0, 0, 0] = 254.0
    real, sc = ref.append_pages(rows, [0, 1], [2], np.array([[0]]), 16, codes, np.ones((1, 1), dtype=np.float32))
    assert sc[0, 0] == 2.0 and np.all(real[0, 0, :2] == 50) and real[0, 0, 2, 0] == 127
    assert np.isnan(real[0, 0, 3:]).all()
    # one visible key: its value; a row before position 0: zeros
    rng = np.random.default_rng(1)
    arrays = ref.make_pool(rng, 1, 1, 16, 64)
    o, _ = ref.attend(rng.standard_normal((2, 1, 64)), [0, 2], [1], arrays, np.array([[0]]), 16, 1.0)
    assert not o[0].any()
    assert np.allclose(o[1, 0], arrays[2][0, 0, 0] * arrays[3][0, 0].astype(np.float64))
