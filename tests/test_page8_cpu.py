"""Plans over a page-scaled FP8 cache: refusals, and work lists that cover
every (row, head, visible key) once. No kernel is launched."""
import numpy as np
import pytest

from paged_kv_attention_27_gb300 import binding as B

from . import _page8
from ._gpu import ensure_built

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    return B.lib()


def _status(f, *a, **kw):
    with pytest.raises(B.FiError) as e:
        f(*a, **kw)
    return e.value.status


def test_both_modes_plan_and_shared_prefixes_do_not():
    opt = {"kv_dtype": B.FI_DTYPE_E4M3_PAGE}
    B.fi_plan(B.FI_MODE_DECODE, 2, None, [0, 2, 3], [5, 16], 8, 2, 128, 16, 0, opt, 4)
    B.fi_plan(B.FI_MODE_PREFILL, 2, [0, 3, 4], [0, 2, 3], [5, 16], 8, 2, 128, 16, 1, opt, 4)
    opt["dtype"] = B.FI_DTYPE_FP16
    B.fi_plan(B.FI_MODE_PREFILL, 2, [0, 3, 4], [0, 2, 3], [5, 16], 8, 2, 128, 16, 1, opt, 4)
    opt.update(prefix_group_indptr=[0, 2], prefix_pages=[1])
    assert _status(B.fi_plan, B.FI_MODE_DECODE, 2, None, [0, 2, 3], [5, 16], 8, 2, 128, 16, 0, opt,
                   4) == B.FI_ERR_UNSUPPORTED
    assert _status(B.fi_plan, B.FI_MODE_DECODE, 1, None, [0, 1], [5], 8, 2, 128, 16, 0,
                   {"dtype": B.FI_DTYPE_E4M3_PAGE}, 4) == B.FI_ERR_INVALID_ARG


def test_page_scales_are_required():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("uses fake device addresses; only meaningful without a GPU")
    opt = {"kv_dtype": B.FI_DTYPE_E4M3_PAGE}
    p = B.fi_plan(B.FI_MODE_DECODE, 2, None, [0, 2, 3], [5, 16], 8, 2, 128, 16, 0, opt, 4)
    args = [p, FAKE, FAKE, FAKE, B.FI_LAYOUT_NHD, 0, 4, FAKE, FAKE, FAKE, 0.1, 1.0, 1.0, FAKE, FAKE, FAKE]
    for kw, st in (({}, B.FI_ERR_INVALID_ARG), ({"k_head_scale": FAKE}, B.FI_ERR_INVALID_ARG),
                   ({"v_head_scale": FAKE}, B.FI_ERR_INVALID_ARG),
                   ({"k_head_scale": FAKE, "v_head_scale": FAKE + 2}, B.FI_ERR_INVALID_ARG),
                   ({"k_head_scale": FAKE, "v_head_scale": FAKE}, B.FI_ERR_NO_DEVICE)):
        assert _status(B.fi_batch_decode_paged, *args, stream=0, **kw) == st
    args[5] = 4104     # a page stride that is no multiple of 16 bytes
    assert _status(B.fi_batch_decode_paged, *args, stream=0, k_head_scale=FAKE,
                   v_head_scale=FAKE) == B.FI_ERR_INVALID_ARG


@pytest.mark.parametrize("seed", range(25))
def test_work_lists_cover_every_row_and_key_once(seed):
    rng = np.random.default_rng(seed)
    g, hkv = int(rng.choice([1, 2, 4, 8])), int(rng.integers(1, 4))
    d, P = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32]))
    n = int(rng.integers(1, 7))
    kv = rng.integers(0, int(rng.choice([20, 700, 6000])), n)
    qo = np.minimum(kv, rng.integers(0, int(rng.choice([3, 40, 600])), n))
    causal = bool(rng.integers(0, 2))
    window = int(rng.choice([-1, -1, 5, 300]))
    b = _page8.Batch(kv, g * hkv, hkv, d, P, qo_lens=qo, causal=causal, window=window, seed=seed)
    plan = b.plan(B, int(rng.choice([1, 20, 152, 1000])))
    info, work = B.fi_plan_get_info(plan), B.fi_plan_get_work(plan)
    rows_per = (256 if d <= 128 else 128) // g
    tile = 128 if d <= 128 else 64
    seen = {}
    for x, (req, head, pb, npg, t0, t1, slot, row) in enumerate(work.tolist()):
        decode = x < info["num_decode_items"]
        a = t0 - t0 % P
        if t1 > t0:
            assert pb == b.page_indptr[req] + a // P and npg == -(-(t1 - a) // P)
        if not decode:
            assert t0 % P == 0 and qo[req] >= 1
            assert (row - b.qo_indptr[req]) % rows_per == 0
        m = 1 if decode else min(rows_per, int(b.qo_indptr[req + 1]) - row)
        for i in range(m):
            pos = kv[req] - qo[req] + (row - b.qo_indptr[req]) + i
            last = pos if (causal or False) else kv[req] - 1
            first = max(0, pos - window) if window >= 0 else 0
            for t in range(max(t0, first), min(t1, last + 1)):
                key = (row + i, head, t)
                seen[key] = seen.get(key, 0) + 1
        if not decode and slot >= 0:      # a piece: whole tiles, but for the last
            assert (t1 - t0) % tile == 0 or t1 <= kv[req]
    want = 0
    for r in range(n):
        for i in range(qo[r]):
            pos = kv[r] - qo[r] + i
            last = pos if causal else kv[r] - 1
            first = max(0, pos - window) if window >= 0 else 0
            want += max(0, last + 1 - first) * hkv
    assert len(seen) == want and all(c == 1 for c in seen.values())


def test_single_rows_beside_a_prefill():
    """Few and short ones are prefill items; many, or one longer than any prefill
    request, stay decode work, and so do those of a batch without longer rows."""
    def decode_items(kv, qo):
        b = _page8.Batch(kv, 8, 2, 64, 16, qo_lens=qo, seed=1)
        info = B.fi_plan_get_info(b.plan(B, 20))
        assert info["num_decode_items"] + info["num_prefill_items"] > 0
        return info["num_decode_items"]
    assert decode_items([500, 400, 500], [5, 1, 1]) == 0
    assert decode_items([500, 501], [5, 1]) > 0
    assert decode_items([2000] + [1900] * 3, [5] + [1] * 3) > 0     # 3 * 15 tiles * 2 heads > 4 * 20
    assert decode_items([2000] + [1900] * 2, [5] + [1] * 2) == 0
    assert decode_items([40, 30, 0], [1, 1, 0]) > 0
