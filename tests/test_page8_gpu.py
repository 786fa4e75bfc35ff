"""Attention over a page-scaled FP8 cache on the GPU against a plain float64
implementation (the bounds are derived in _page8.py)."""
import numpy as np
import pytest

from paged_kv_attention_27_gb300 import binding as B

from . import _page8
from ._gpu import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    return B.lib()


def _check(b, sms=None, what="", **kw):
    d = _page8.Device(b, sms)
    out, lse = d.run(**kw)
    assert d.status() == B.FI_OK
    _page8.compare(b, out, lse, _page8.reference(b, **kw), what=what)
    return d


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 300, 700, 0, 45]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("layout,P,dtype", [("NHD", 16, "bf16"), ("HND", 32, "bf16"),
                                            ("HND", 16, "fp16"), ("NHD", 32, "fp16")])
def test_decode_shapes(d, g, layout, P, dtype):
    b = _page8.Batch(LENS, 2 * g, 2, d, P, layout, dtype, seed=d + g, tail=0x7f)
    _check(b, what=f"d{d} g{g} {layout} {dtype}")


@pytest.mark.parametrize("sms", [1, 3, 152, 2000])
@pytest.mark.parametrize("g,d", [(8, 128), (1, 64), (4, 256)])
def test_decode_splits(sms, g, d):
    b = _page8.Batch([5000, 1, 1300, 2049, 0, 640], 2 * g, 2, d, 16, seed=7)
    _check(b, sms, what=f"sms {sms}")


@pytest.mark.parametrize("w", [0, 1, 15, 16, 17, 127, 128, 300, 5000])
@pytest.mark.parametrize("g,d", [(8, 128), (2, 64), (1, 256)])
def test_decode_window(w, g, d):
    b = _page8.Batch([1, 16, 40, 333, 1500], 2 * g, 2, d, 16, window=w, seed=w, tail=0xff)
    # keys before the window, on its first page too, hold NaN codes
    for r, n in enumerate(b.kv_lens):
        for t in range(max(0, n - 1 - w)):
            page = b.page_indices[b.page_indptr[r] + t // 16]
            for c in b.codes:
                c[page, t % 16] = 0x7f
    ref_b = _page8.Batch([1, 16, 40, 333, 1500], 2 * g, 2, d, 16, window=w, seed=w)
    dv = _page8.Device(b)
    out, lse = dv.run()
    assert dv.status() == B.FI_OK
    _page8.compare(b, out, lse, _page8.reference(ref_b), what=f"window {w}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("g,d", [(8, 128), (1, 128), (4, 64), (2, 256)])
def test_decode_any_scales(g, d, dtype):
    """Scales that are no powers of two, and pages whose values (and so their
    scales) differ by 2^24; tensor-wide scales on top."""
    b = _page8.Batch([900, 33, 257], 2 * g, 2, d, 16, dtype=dtype, seed=3, scales="any")
    _check(b, what="any", k_scale=0.5, v_scale=3.0)
    b = _page8.Batch([900, 33, 257], 2 * g, 2, d, 16, seed=4, v_spread=12)
    _check(b, what="spread")


def test_decode_small_scale_pages_keep_their_weight():
    """The page with all the weight has values 2^40 times smaller than the
    others': its own values have to come out."""
    import torch
    b = _page8.Batch([64], 8, 1, 128, 16, seed=5)
    b.codes[0][:] = 0x38                      # every key element 1
    for s in b.scale:
        s[:] = 1.0
    b.scale[0][b.page_indices[2], 0] = 64.0   # keys of page 2: 64
    b.scale[1][b.page_indices[2], 0] = 2.0 ** -40
    b.q = torch.ones_like(b.q)
    _check(b, what="small page")


def test_decode_q_range_and_special_values():
    """q elements over fp16's and bf16's whole range of a row, a zero row, and
    rows with a NaN or an infinity, which stay their own."""
    import torch
    for dtype, lo in (("bf16", -30), ("fp16", -12)):
        b = _page8.Batch([200] * 6, 4, 1, 128, 16, dtype=dtype, seed=6)
        e = torch.from_numpy(np.random.default_rng(1).integers(lo, 1, (6, 4, 128)))
        b.q = (b.q.double() * torch.exp2(e.double())).to(b.q.dtype)
        b.q[1] = 0
        _check(b, what=f"range {dtype}")
        b.q[2, 1, 5] = float("nan")
        b.q[3, 2, 7] = float("inf")
        d = _page8.Device(b)
        out, lse = d.run()
        bad = torch.isnan(out).all(dim=2).cpu().numpy()
        want = np.zeros((6, 4), dtype=bool)
        want[2, 1] = want[3, 2] = True
        assert np.array_equal(bad, want) and np.array_equal(torch.isnan(lse).cpu().numpy(), want)
        assert np.array_equal(torch.isnan(out).any(dim=2).cpu().numpy(), want)


def test_decode_sm_scale_zero_is_the_mean():
    b = _page8.Batch([70, 16, 129], 8, 2, 64, 16, seed=8)
    b.sm_scale = 0.0
    _check(b, what="mean")


def test_decode_deterministic_and_without_lse():
    import torch
    b = _page8.Batch([3000, 50, 900, 2000], 16, 2, 128, 16, seed=9)
    d = _page8.Device(b, 40)
    o1, l1 = [x.clone() for x in d.run()]
    for _ in range(3):
        d.out.fill_(7)
        o2, l2 = d.run()
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    d.lse.fill_(-3)
    d.run(lse=False)
    assert torch.equal(d.out, o1) and bool((d.lse == -3).all())


def test_decode_page_views_of_one_buffer():
    import torch
    b = _page8.Batch([100, 40], 8, 2, 128, 16, seed=10)
    d = _page8.Device(b)
    o1 = d.run()[0].clone()
    kv = torch.zeros(b.num_pages, 2, 16, 2, 128, dtype=torch.uint8, device="cuda")
    kv[:, 0], kv[:, 1] = d.k, d.v
    d.k, d.v = kv, kv[:, 1]
    d.out.zero_()
    assert torch.equal(d.run(page_stride=2 * 16 * 2 * 128)[0], o1)


def test_decode_page_outside_the_cache_is_skipped_and_reported():
    b = _page8.Batch([100, 60], 8, 2, 128, 16, seed=11)
    d = _page8.Device(b)
    want = _page8.reference(b)
    d.page_indices[2] = b.num_pages
    d.page_indices[3] = -1
    out, lse = d.run()
    assert d.status() == B.FI_ERR_DEVICE_BOUNDS
    rows = np.array([1])
    _page8.compare(b, out, lse, want, rows=rows, what="other request")
    # the request itself: its keys without the two pages
    q, k, v = b.q64()[0], b.kv64(0), b.kv64(1)
    t = np.array([x for x in range(100) if x // 16 not in (2, 3)])
    pages = b.page_indices[t // 16]
    for h in range(8):
        s = b.sm_scale * (k[pages, t % 16, h // 4] @ q[h])
        p = np.exp(s - s.max())
        o = p @ v[pages, t % 16, h // 4] / p.sum()
        assert np.abs(out[0, h].double().cpu().numpy() - o).max() < 2e-2
        assert abs(lse[0, h].item() - (s.max() + np.log(p.sum()))) < 1e-4
    d.page_indices[2], d.page_indices[3] = int(b.page_indices[2]), int(b.page_indices[3])
    _page8.compare(b, *d.run(), want, what="after")
    assert d.status() == B.FI_OK


@pytest.mark.parametrize("d,g", [(128, 8), (64, 1), (256, 4)])
def test_decode_bounded_wait_and_recovery(d, g):
    b = _page8.Batch([300, 40, 1000], 2 * g, 2, d, 16, seed=12)
    dv = _page8.Device(b)
    B.fi_debug_set_fault(1, 50_000_000)
    try:
        dv.run()
        assert dv.status() == B.FI_ERR_DEVICE_TIMEOUT
    finally:
        B.fi_debug_set_fault(0, 0)
    _page8.compare(b, *dv.run(), _page8.reference(b), what="after")
    assert dv.status() == B.FI_OK


def test_decode_through_host_buffers_and_without_workspace():
    import torch
    b = _page8.Batch([500, 3, 0, 64], 8, 2, 128, 16, seed=13)
    d = _page8.Device(b)
    o1, l1 = [x.clone() for x in d.run()]
    d.out.zero_()
    B.fi_batch_decode_paged_noalloc(d.plan, d.q, d.k, d.v, B.FI_LAYOUT_NHD, 0, b.num_pages,
                                    d.page_indptr, d.page_indices, d.last_page_len, b.sm_scale, 1.0,
                                    1.0, d.out, d.lse, k_head_scale=d.ks, v_head_scale=d.vs)
    torch.cuda.synchronize()
    assert torch.equal(d.out, o1) and torch.equal(d.lse, l1)
    info = B.fi_plan_get_info(d.plan)
    ws = torch.empty(info["workspace_bytes"] + info["host_io_bytes"], dtype=torch.uint8, device="cuda")
    oh, lh = torch.empty(o1.shape, dtype=o1.dtype), torch.empty(l1.shape)
    B.fi_batch_attention_host(d.plan, b.q.contiguous(), None, d.k, d.v, B.FI_LAYOUT_NHD, 0,
                              b.num_pages, b.page_indptr, b.page_indices, b.last_page_len,
                              b.sm_scale, 1.0, 1.0, oh, lh, ws, ws.numel(), k_head_scale=d.ks,
                              v_head_scale=d.vs)
    assert torch.equal(oh, o1.cpu()) and torch.equal(lh, l1.cpu())


def test_decode_on_another_stream():
    import torch
    b = _page8.Batch([2000, 64, 333], 8, 2, 128, 16, seed=14)
    d = _page8.Device(b)
    o1 = d.run()[0].clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        d.out.zero_()
        d.run()
    s.synchronize()
    assert torch.equal(d.out, o1)


# ---- prefill -----------------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("layout,P,dtype", [("NHD", 16, "bf16"), ("HND", 32, "fp16")])
def test_prefill_shapes(d, g, layout, P, dtype):
    """Whole prompts, chunks on earlier keys, a few rows, single rows, empty
    requests; row counts that end inside a tile and at its edge."""
    kv = [5, 300, 1, 0, 129, 70, 700, 64, 257, 33]
    qo = [5, 300, 1, 0, 1, 3, 130, 33, 257, 0]
    b = _page8.Batch(kv, 2 * g, 2, d, P, layout, dtype, qo_lens=qo, seed=d + g, tail=0x7f)
    _check(b, what=f"d{d} g{g} {layout} {dtype}")


@pytest.mark.parametrize("g,d", [(8, 128), (1, 64), (2, 256)])
def test_prefill_not_causal(g, d):
    b = _page8.Batch([40, 0, 300, 129], 2 * g, 2, d, 16, qo_lens=[70, 4, 9, 1], causal=False, seed=21,
                     tail=0xff)
    _check(b, what="full")


@pytest.mark.parametrize("sms", [1, 152, 2000])
@pytest.mark.parametrize("g,d", [(8, 128), (4, 64), (2, 256)])
def test_prefill_splits(sms, g, d):
    b = _page8.Batch([5000, 3000, 900], 2 * g, 2, d, 16, qo_lens=[60, 7, 140], seed=22)
    assert (B.fi_plan_get_info(b.plan(B, sms))["num_partial_slots"] > 0) == (sms > 1)
    _check(b, sms, what=f"sms {sms}")


@pytest.mark.parametrize("w", [0, 1, 16, 100, 127, 128, 1000])
@pytest.mark.parametrize("g,d", [(8, 128), (1, 64), (4, 256)])
def test_prefill_window(w, g, d):
    b = _page8.Batch([333, 40, 900], 2 * g, 2, d, 16, qo_lens=[333, 3, 50], window=w, seed=w)
    _check(b, what=f"window {w}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("g,d", [(8, 128), (1, 128), (4, 64), (2, 256)])
def test_prefill_any_scales(g, d, dtype):
    kv, qo = [900, 33, 257], [40, 33, 200]
    b = _page8.Batch(kv, 2 * g, 2, d, 16, dtype=dtype, qo_lens=qo, seed=3, scales="any")
    _check(b, what="any", k_scale=0.5, v_scale=3.0)
    b = _page8.Batch(kv, 2 * g, 2, d, 32, qo_lens=qo, seed=4, v_spread=12)
    _check(b, what="spread")


def test_prefill_small_scale_pages_keep_their_weight():
    import torch
    b = _page8.Batch([64], 8, 1, 128, 16, qo_lens=[16], seed=5)
    b.codes[0][:] = 0x38
    for s in b.scale:
        s[:] = 1.0
    b.scale[0][b.page_indices[2], 0] = 64.0
    b.scale[1][b.page_indices[2], 0] = 2.0 ** -40
    b.q = torch.ones_like(b.q)
    _check(b, what="small page")


def test_prefill_q_range_and_special_values():
    import torch
    for dtype, lo in (("bf16", -30), ("fp16", -12)):
        b = _page8.Batch([200, 90], 4, 1, 128, 16, dtype=dtype, qo_lens=[30, 40], seed=6)
        e = torch.from_numpy(np.random.default_rng(1).integers(lo, 1, (70, 4, 128)))
        b.q = (b.q.double() * torch.exp2(e.double())).to(b.q.dtype)
        b.q[1] = 0
        _check(b, what=f"range {dtype}")
        b.q[2, 1, 5] = float("nan")
        b.q[50, 2, 7] = float("inf")
        d = _page8.Device(b)
        out, lse = d.run()
        want = np.zeros((70, 4), dtype=bool)
        want[2, 1] = want[50, 2] = True
        assert np.array_equal(torch.isnan(out).all(dim=2).cpu().numpy(), want)
        assert np.array_equal(torch.isnan(out).any(dim=2).cpu().numpy(), want)
        assert np.array_equal(torch.isnan(lse).cpu().numpy(), want)


def test_prefill_deterministic_rows_behind_stay():
    import torch
    b = _page8.Batch([3000, 500, 900], 16, 2, 128, 16, qo_lens=[300, 2, 77], seed=9)
    d = _page8.Device(b)
    out = torch.full((b.rows + 5, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    d.out = out[:b.rows]
    o1, l1 = [x.clone() for x in d.run()]
    assert bool((out[b.rows:] == 7).all())
    for _ in range(3):
        d.out.fill_(7)
        o2, l2 = d.run()
        assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_prefill_page_outside_the_cache_is_skipped_and_reported():
    b = _page8.Batch([200, 60], 8, 2, 128, 16, qo_lens=[20, 10], seed=11)
    d = _page8.Device(b)
    want = _page8.reference(b)
    d.page_indices[2] = b.num_pages
    d.page_indices[3] = -1
    out, lse = d.run()
    assert d.status() == B.FI_ERR_DEVICE_BOUNDS
    _page8.compare(b, out, lse, want, rows=np.arange(20, 30), what="other request")
    q, k, v = b.q64(), b.kv64(0), b.kv64(1)
    for i in (0, 19):
        t = np.array([x for x in range(181 + i) if x // 16 not in (2, 3)])
        pages = b.page_indices[t // 16]
        for h in (0, 7):
            s = b.sm_scale * (k[pages, t % 16, h // 4] @ q[i, h])
            p = np.exp(s - s.max())
            o = p @ v[pages, t % 16, h // 4] / p.sum()
            assert np.abs(out[i, h].double().cpu().numpy() - o).max() < 2e-2
            assert abs(lse[i, h].item() - (s.max() + np.log(p.sum()))) < 1e-4
    d.page_indices[2], d.page_indices[3] = int(b.page_indices[2]), int(b.page_indices[3])
    _page8.compare(b, *d.run(), want, what="after")
    assert d.status() == B.FI_OK


@pytest.mark.parametrize("d,g", [(128, 8), (64, 1), (256, 4)])
def test_prefill_bounded_wait_and_recovery(d, g):
    b = _page8.Batch([300, 40, 1000], 2 * g, 2, d, 16, qo_lens=[100, 2, 1], seed=12)
    dv = _page8.Device(b)
    B.fi_debug_set_fault(1, 50_000_000)
    try:
        dv.run()
        assert dv.status() == B.FI_ERR_DEVICE_TIMEOUT
    finally:
        B.fi_debug_set_fault(0, 0)
    _page8.compare(b, *dv.run(), _page8.reference(b), what="after")
    assert dv.status() == B.FI_OK


def test_prefill_through_host_buffers():
    import torch
    b = _page8.Batch([500, 3, 0, 64], 8, 2, 128, 16, qo_lens=[200, 3, 0, 1], seed=13)
    d = _page8.Device(b)
    o1, l1 = [x.clone() for x in d.run()]
    info = B.fi_plan_get_info(d.plan)
    ws = torch.empty(info["workspace_bytes"] + info["host_io_bytes"], dtype=torch.uint8, device="cuda")
    oh, lh = torch.empty(o1.shape, dtype=o1.dtype), torch.empty(l1.shape)
    B.fi_batch_attention_host(d.plan, b.q.contiguous(), b.qo_indptr, d.k, d.v, B.FI_LAYOUT_NHD, 0,
                              b.num_pages, b.page_indptr, b.page_indices, b.last_page_len,
                              b.sm_scale, 1.0, 1.0, oh, lh, ws, ws.numel(), k_head_scale=d.ks,
                              v_head_scale=d.vs)
    assert torch.equal(oh, o1.cpu()) and torch.equal(lh, l1.cpu())


@pytest.mark.parametrize("g,d,dtype", [(8, 128, "bf16"), (2, 64, "bf16"), (4, 256, "fp16"),
                                       (1, 128, "fp16")])
def test_prefill_many_items_of_few_keys(g, d, dtype):
    """Thousands of items with one K/V tile or none, next to each other, with
    one and with two row tiles: the pipeline's phases move from item to item
    with nothing in between. Every pass ends, without a wait that ran out, and
    gives the same bits."""
    import torch
    rng = np.random.default_rng(31)
    kv = rng.integers(1, 129, 300)
    kv[::7] = rng.integers(100, 300, len(kv[::7]))
    qo = np.minimum(kv, rng.integers(2, 2 * 256 // g, 300))
    b = _page8.Batch(kv, 8 * g, 8, d, 16, dtype=dtype, qo_lens=qo, seed=31)
    dv = _page8.Device(b)
    o1, l1 = [x.clone() for x in dv.run()]
    some = [0, 7, 50, 299]
    rows = np.concatenate([np.arange(b.qo_indptr[r], b.qo_indptr[r + 1]) for r in some])
    _page8.compare(b, o1, l1, _page8.reference(b, some), rows=rows, what="some")
    assert dv.status() == B.FI_OK
    for _ in range(100):
        dv.run()
        assert torch.equal(dv.out, o1) and torch.equal(dv.lse, l1)
        assert dv.status() == B.FI_OK


def test_prefill_many_items_without_keys():
    """Rows of requests without keys between others (not causal): zeros."""
    import torch
    kv = [0, 0, 50, 0, 0, 0, 300, 0] * 20
    b = _page8.Batch(kv, 8, 2, 128, 16, qo_lens=[3, 70, 5, 9, 2, 200, 40, 2] * 20, causal=False, seed=32)
    dv = _page8.Device(b)
    o1, l1 = [x.clone() for x in dv.run()]
    _page8.compare(b, o1, l1, _page8.reference(b), what="empty")
    for _ in range(50):
        dv.run()
        assert torch.equal(dv.out, o1) and dv.status() == B.FI_OK


@pytest.mark.parametrize("g,d,dtype", [(8, 128, "bf16"), (1, 64, "bf16"), (4, 256, "fp16")])
def test_decode_many_items_of_few_keys(g, d, dtype):
    """Thousands of items with one tile, a few or none next to each other: the
    same bits in every pass, and no wait that ran out."""
    import torch
    rng = np.random.default_rng(33)
    kv = rng.integers(0, 130, 700)
    kv[::9] = rng.integers(100, 700, len(kv[::9]))
    b = _page8.Batch(kv, 4 * g, 4, d, 16, dtype=dtype, seed=33)
    dv = _page8.Device(b)
    o1, l1 = [x.clone() for x in dv.run()]
    some = [0, 9, 50, 699]
    _page8.compare(b, o1, l1, _page8.reference(b, some), rows=np.array(some), what="some")
    for _ in range(100):
        dv.run()
        assert torch.equal(dv.out, o1) and torch.equal(dv.lse, l1)
        assert dv.status() == B.FI_OK


def test_decode_nan_rows_of_split_requests_stay_nan():
    import torch
    b = _page8.Batch([3000, 5000, 40], 8, 2, 128, 16, seed=34)
    _check(b, 152, what="split")
    b.q[0, 1, 5] = float("nan")
    b.q[1, 6, 0] = float("inf")
    d = _page8.Device(b, 152)
    assert B.fi_plan_get_info(d.plan)["num_split_requests"] == 2
    out, lse = d.run()
    want = np.zeros((3, 8), dtype=bool)
    want[0, 1] = want[1, 6] = True
    assert np.array_equal(torch.isnan(out).all(dim=2).cpu().numpy(), want)
    assert np.array_equal(torch.isnan(out).any(dim=2).cpu().numpy(), want)
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), want)


def test_prefill_nan_rows_of_split_items_stay_nan():
    import torch
    b = _page8.Batch([5000], 8, 2, 128, 16, qo_lens=[20], seed=35)
    assert B.fi_plan_get_info(b.plan(B, 152))["num_partial_slots"] > 0
    b.q[3, 1, 5] = float("nan")
    b.q[19, 6, 0] = float("inf")
    d = _page8.Device(b, 152)
    out, lse = d.run()
    want = np.zeros((20, 8), dtype=bool)
    want[3, 1] = want[19, 6] = True
    assert np.array_equal(torch.isnan(out).all(dim=2).cpu().numpy(), want)
    assert np.array_equal(torch.isnan(out).any(dim=2).cpu().numpy(), want)
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), want)


# ---- both ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("g,d,P", [(8, 128, 16), (1, 64, 32), (4, 256, 16)])
def test_value_scales_2_80_apart(g, d, P, prefill):
    """Neighbouring pages' V scales differ by the documented 2^80, the first
    page's being the smaller or the larger one."""
    b = _page8.Batch([500, 70, 16], 2 * g, 2, d, P, qo_lens=[30, 70, 5] if prefill else None, seed=16)
    up = np.arange(len(b.page_indices)) % 2 == 0
    b.scale[1][b.page_indices[up]] *= 2.0 ** 40
    b.scale[1][b.page_indices[~up]] *= 2.0 ** -40
    _check(b, what="2^80 apart")


@pytest.mark.parametrize("prefill", [False, True])
def test_two_streams_at_once_with_one_plan(prefill):
    import torch
    qo = [200, 1, 17, 300] if prefill else None
    b = _page8.Batch([3000, 64, 333, 1800], 16, 2, 128, 16, qo_lens=qo, seed=17)
    x, y = _page8.Device(b), _page8.Device(b)
    y.plan = x.plan
    want = x.run()[0].clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for d, s in zip((x, y), streams):
            with torch.cuda.stream(s):
                d.out.fill_(7)
                d.run()
    torch.cuda.synchronize()
    for d in (x, y):
        assert d.status() == B.FI_OK and torch.equal(d.out, want)


def test_cache_offsets_beyond_32_bits():
    """Pages 2^28 bytes apart: append to and attention over a cache whose offsets
    pass 2^32."""
    import torch
    P, H, d = 16, 2, 128
    stride = 1 << 28
    buf = torch.empty(18 * stride, dtype=torch.uint8, device="cuda")
    for qo in (None, [40, 9]):
        b = _page8.Batch([170, 60], 8, H, d, P, qo_lens=qo, seed=18, spare=2)
        assert b.num_pages * stride > 1 << 32
        x = _page8.Device(b)
        k = buf.as_strided((b.num_pages, P, H, d), (stride, H * d, d, 1))
        v = k.as_strided(k.shape, k.stride(), storage_offset=1 << 20)
        # the last keys of request 0 come by an append
        page = int(b.page_indices[b.page_indptr[1] - 1])
        n = int(b.last_page_len[0])
        k.copy_(x.k)
        v.copy_(x.v)
        k[page], v[page] = 0, 0
        ws = torch.zeros(B.FI_STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        kn, vn = [(torch.from_numpy(b.kv64(i)[page, :n]).to(torch.bfloat16)).cuda() for i in (0, 1)]
        smap = torch.arange(page * P, page * P + n, device="cuda")
        B.fi_append_paged_kv(n, smap, kn, vn, 0, B.FI_DTYPE_BF16, H, d, k, v, B.FI_DTYPE_E4M3_PAGE,
                             B.FI_LAYOUT_NHD, stride, b.num_pages, P, x.ks, x.vs, ws)
        assert B.fi_check_device_status(ws) == B.FI_OK
        b.scale[0][page], b.scale[1][page] = x.ks[page].cpu().numpy(), x.vs[page].cpu().numpy()
        b.codes[0][page], b.codes[1][page] = k[page].cpu().numpy(), v[page].cpu().numpy()
        assert b.codes[0][page, :n].any() and not b.codes[0][page, n:].any()
        x.k, x.v = k, v
        out, lse = x.run(page_stride=stride)
        assert x.status() == B.FI_OK
        _page8.compare(b, out, lse, _page8.reference(b), what="far pages")


def test_calls_back_to_back_in_one_workspace():
    """Launches may start beside the ones in front of them: appends, small and
    large plans of both modes, copies into q and out of the results, all in one
    stream and workspace with nothing between them, against the same calls one
    at a time."""
    import torch
    P, H, d = 16, 2, 128
    shapes = [([300, 40], None), ([2000] * 60, None), ([700, 30], [90, 3]), ([900] * 12, [5] * 12),
              ([5], None), ([4000], [600])]
    batches = [_page8.Batch(kv, 8, H, d, P, qo_lens=qo, seed=20 + i) for i, (kv, qo) in enumerate(shapes)]
    ws_bytes = max(_page8.Device(b).plan.workspace_bytes for b in batches)
    step_ws = torch.zeros(B.FI_STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    rounds = 6
    new = torch.randn(rounds, 8, 2 * H, d, device="cuda", generator=g).to(torch.bfloat16)
    smap = [torch.arange(8, device="cuda") + int(b.page_indices[0]) * P for b in batches]

    def go(wait):
        ws = torch.zeros(ws_bytes, dtype=torch.uint8, device="cuda")
        devs = [_page8.Device(b) for b in batches]
        for x in devs:
            x.workspace = ws
        torch.cuda.synchronize()
        outs = []
        for r in range(rounds):
            for x, m in zip(devs, smap):
                # the first 8 keys of request 0 anew, then attention, then q from its result
                B.fi_append_paged_kv(min(8, x.b.kv_lens[0]), m, new[r, :, :H], new[r, :, H:], 2 * H * d,
                                     B.FI_DTYPE_BF16, H, d, x.k, x.v, B.FI_DTYPE_E4M3_PAGE,
                                     B.FI_LAYOUT_NHD, 0, x.b.num_pages, P, x.ks, x.vs, step_ws)
                if wait:
                    torch.cuda.synchronize()
                x.run()
                if wait:
                    torch.cuda.synchronize()
                outs.append((x.out.clone(), x.lse.clone()))
                x.q.add_(x.out)
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert B.fi_check_device_status(ws) == B.FI_OK
        return outs

    want = go(True)
    for _ in range(3):
        for (o, l), (wo, wl) in zip(go(False), want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_a_call_waits_for_both_streams_of_a_mixed_one():
    """A mixed batch runs its decode rows on a side stream; the next call, in the
    same workspace, comes after both. (The second plan is the smaller one in
    every way.)"""
    import torch
    kv, qo = [400, 90] + [6000] * 24, [120, 90] + [1] * 24
    x = _page8.Device(_page8.Batch(kv, 8, 2, 128, 16, qo_lens=qo, seed=30))
    y = _page8.Device(_page8.Batch([70, 5], 8, 2, 128, 16, seed=31))
    assert y.plan.workspace_bytes <= x.plan.workspace_bytes
    y.workspace = x.workspace
    want = []
    for d in (x, y):
        want.append([t.clone() for t in d.run()])
        assert d.status() == B.FI_OK
    for _ in range(30):
        x.out.fill_(7)
        y.out.fill_(7)
        x.run()
        y.run()
        torch.cuda.synchronize()
        for d, (o, l) in zip((x, y), want):
            assert torch.equal(d.out, o) and torch.equal(d.lse, l)
    assert x.status() == B.FI_OK
