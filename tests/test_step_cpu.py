"""Refusals of the step calls (page tables, append) and of page-scaled plans,
and pins of the plain implementations the GPU tests compare with. No kernel
is launched."""
import numpy as np
import pytest

from paged_kv_attention_27_gb300 import binding as B

from . import _step
from ._gpu import ensure_built

FAKE = 1 << 20   # aligned, never dereferenced: every call below returns first


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    return B.lib()


def _no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("uses fake device addresses; only meaningful without a GPU")


def _status(call, args, **kw):
    with pytest.raises(B.FiError) as e:
        call(*args, stream=0, **kw)
    return e.value.status


STEP = dict(batch=2, slots=FAKE, new_len=FAKE, max_requests=4, max_pages=8, page_size=16,
            kv_len=FAKE, kv_len_out=FAKE, block_table=FAKE, free_ring=FAKE, ring_capacity=32,
            ring_state=FAKE, ring_state_out=FAKE, page_indptr=FAKE, page_indices=FAKE,
            page_capacity=16, last_page_len=FAKE, qo_indptr=FAKE, slot_map=FAKE, positions=FAKE,
            token_capacity=64, workspace=FAKE, workspace_bytes=256)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=8193), dict(max_requests=0), dict(max_requests=262145),
    dict(max_pages=0), dict(page_size=0), dict(page_size=1025), dict(ring_capacity=0),
    dict(page_capacity=-1), dict(token_capacity=-1), dict(new_len=None), dict(kv_len=None),
    dict(kv_len_out=None), dict(block_table=None), dict(free_ring=None), dict(ring_state=None),
    dict(ring_state_out=None), dict(page_indptr=None), dict(page_indices=None),
    dict(last_page_len=None), dict(qo_indptr=None), dict(slot_map=None), dict(workspace=None),
    dict(slots=FAKE + 2), dict(slot_map=FAKE + 4), dict(workspace=FAKE + 128),
    dict(positions=FAKE + 1)])
def test_page_table_step_refusals(bad):
    _no_gpu()
    args = {**STEP, **bad}
    assert _status(lambda **k: B.fi_page_table_step(**args, **k), ()) == B.FI_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["ring_capacity", "page_capacity", "token_capacity"])
def test_page_table_step_capacity_limit(name):
    _no_gpu()
    for n, status in ((2 ** 30, B.FI_ERR_NO_DEVICE), (2 ** 30 + 1, B.FI_ERR_INVALID_ARG)):
        assert _status(lambda **k: B.fi_page_table_step(**{**STEP, name: n}, **k), ()) == status


def test_page_table_step_accepts_what_it_documents():
    _no_gpu()
    call = lambda **kw: _status(lambda **k: B.fi_page_table_step(**{**STEP, **kw}, **k), ())
    assert call(workspace_bytes=255) == B.FI_ERR_WORKSPACE_TOO_SMALL
    for kw in ({}, dict(slots=None), dict(positions=None), dict(page_capacity=0, page_indices=None),
               dict(token_capacity=0, slot_map=None, positions=None), dict(batch=8192),
               dict(max_requests=262144)):
        assert call(**kw) == B.FI_ERR_NO_DEVICE, kw
    B.fi_page_table_step(**{**STEP, "batch": 0, "kv_len": None}, stream=0)   # nothing to do


APPEND = dict(num_tokens=3, slot_map=FAKE, k_new=FAKE, v_new=FAKE, token_stride_elems=0,
              dtype=B.FI_DTYPE_BF16, num_kv_heads=2, head_dim=128, k_cache=FAKE, v_cache=FAKE,
              kv_dtype=B.FI_DTYPE_E4M3_PAGE, kv_layout=B.FI_LAYOUT_NHD, page_stride_elems=0,
              num_pages=4, page_size=16, k_page_scale=FAKE, v_page_scale=FAKE, workspace=FAKE,
              workspace_bytes=256)


@pytest.mark.parametrize("bad,status", [
    (dict(num_tokens=-1), B.FI_ERR_INVALID_ARG), (dict(num_kv_heads=0), B.FI_ERR_INVALID_ARG),
    (dict(dtype=B.FI_DTYPE_E4M3), B.FI_ERR_INVALID_ARG),
    (dict(kv_dtype=B.FI_DTYPE_FP16), B.FI_ERR_INVALID_ARG),
    (dict(kv_dtype=7), B.FI_ERR_INVALID_ARG), (dict(kv_layout=2), B.FI_ERR_INVALID_ARG),
    (dict(kv_dtype=B.FI_DTYPE_E4M3), B.FI_ERR_UNSUPPORTED),
    (dict(head_dim=96), B.FI_ERR_UNSUPPORTED), (dict(page_size=64), B.FI_ERR_UNSUPPORTED),
    (dict(token_stride_elems=255), B.FI_ERR_INVALID_ARG),
    (dict(token_stride_elems=260), B.FI_ERR_INVALID_ARG),
    (dict(page_stride_elems=4095), B.FI_ERR_INVALID_ARG),
    (dict(page_stride_elems=4104), B.FI_ERR_INVALID_ARG),
    (dict(slot_map=None), B.FI_ERR_INVALID_ARG), (dict(k_new=None), B.FI_ERR_INVALID_ARG),
    (dict(v_cache=None), B.FI_ERR_INVALID_ARG), (dict(k_page_scale=None), B.FI_ERR_INVALID_ARG),
    (dict(v_page_scale=None), B.FI_ERR_INVALID_ARG), (dict(workspace=None), B.FI_ERR_INVALID_ARG),
    (dict(slot_map=FAKE + 4), B.FI_ERR_INVALID_ARG), (dict(v_new=FAKE + 8), B.FI_ERR_INVALID_ARG),
    (dict(k_cache=FAKE + 8), B.FI_ERR_INVALID_ARG), (dict(k_page_scale=FAKE + 2), B.FI_ERR_INVALID_ARG),
    (dict(workspace_bytes=8), B.FI_ERR_WORKSPACE_TOO_SMALL), ({}, B.FI_ERR_NO_DEVICE),
    (dict(token_stride_elems=1024), B.FI_ERR_NO_DEVICE),
    (dict(page_stride_elems=8192), B.FI_ERR_NO_DEVICE),
    (dict(kv_dtype=B.FI_DTYPE_BF16, k_page_scale=None, v_page_scale=None), B.FI_ERR_NO_DEVICE)])
def test_append_refusals(bad, status):
    _no_gpu()
    args = {**APPEND, **bad}
    assert _status(lambda **k: B.fi_append_paged_kv(**args, **k), ()) == status


def test_append_of_no_rows_does_nothing():
    B.fi_append_paged_kv(**{**APPEND, "num_tokens": 0, "slot_map": None, "k_new": None}, stream=0)


def test_out_of_pages_has_a_status_string():
    assert B.status_string(B.FI_ERR_OUT_OF_PAGES) == "not enough free pages"


# ---- pins of the plain implementations -----------------------------------------------------------
def test_e4m3_codes_against_torch():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_step.e4m3_value(codes), want, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * \
        np.exp2(np.random.default_rng(1).integers(-14, 8, 20000)).astype(np.float32)
    x = np.clip(x, -448, 448)
    x = np.concatenate([x, want[np.isfinite(want)].astype(np.float32),
                        ((want[8:126] + want[9:127]) / 2).astype(np.float32)])   # ties
    got = _step.e4m3_value(_step.e4m3_code(x))
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (449.0, 2.0), (896.0, 2.0),
                                        (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (0.0, 2.0 ** -100),
                                        (1.0, 2.0 ** -8), (2.0 ** -120, 2.0 ** -100)])
def test_scale_is_the_smallest_power_of_two(amax, scale):
    assert _step.scale_of(amax) == scale


def test_page_table_step_closed_form():
    """Two requests and a padding row by hand: 16-token pages."""
    table = np.full((3, 4), -1)
    table[2, 0] = 7                                   # slot 2 has 10 tokens on page 7
    table[0, :2] = [5, 6]                             # slot 0 has 18 tokens
    r = _step.page_table_step([2, -1, 0], [7, 3, -4], np.array([18, 0, 10]), table,
                              np.array([9, 1, 2, 3, 4]), [4, 3], 16, 8, 8)
    assert r["page_indptr"].tolist() == [0, 2, 2, 3]
    assert r["page_indices"].tolist() == [7, 4, 5]    # the ring's head is entry 4
    assert r["last_page_len"].tolist() == [1, 0, 14]
    assert r["qo_indptr"].tolist() == [0, 7, 7, 7]
    assert r["slot_map"].tolist() == [122, 123, 124, 125, 126, 127, 64, -1]
    assert r["positions"].tolist() == [10, 11, 12, 13, 14, 15, 16, 0]
    assert r["kv_len"].tolist() == [14, 0, 17]
    assert r["free_ring"].tolist() == [9, 1, 6, 3, 4]  # page 6 at (4 + 3) % 5
    assert r["ring_state"].tolist() == [0, 3]
