"""The step calls on the GPU against their plain implementations: every
output, and what has to stay as it was. Both calls are exact, so every
comparison is for equality."""
import numpy as np
import pytest

from paged_kv_attention_27_gb300 import binding as B

from . import _step
from ._gpu import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    return B.lib()


def _torch():
    import torch
    return torch


class Server:
    """Requests in slots with their pages, on the host; `step` runs the call
    on copies and returns its arrays."""

    def __init__(self, slots, max_pages, page_size, pool, seed):
        self.rng = np.random.default_rng(seed)
        self.P, self.max_pages = page_size, max_pages
        self.kv_len = np.zeros(slots, dtype=np.int32)
        self.table = np.full((slots, max_pages), -1, dtype=np.int32)
        self.ring = self.rng.permutation(pool).astype(np.int32)
        self.state = np.array([0, pool], dtype=np.int32)

    def fill(self, lens):
        at = 0
        for s, n in enumerate(lens):
            m = -(-n // self.P)
            self.kv_len[s] = n
            self.table[s, :m] = self.ring[at:at + m]
            at += m
        self.ring[:at] = -5                            # taken: not to be read
        self.state[:] = (at % len(self.ring), len(self.ring) - at)

    def step(self, slots, new_len, page_capacity, token_capacity, in_place=True, workspace=None,
             positions=True, null_slots=False):
        torch = _torch()
        dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()
        full = lambda n, t=torch.int32: torch.full((max(n, 1),), -77, dtype=t, device="cuda")
        n = len(slots)
        d = dict(slots=dev(slots), new_len=dev(new_len), kv_len=dev(self.kv_len),
                 block_table=dev(self.table), free_ring=dev(self.ring), ring_state=dev(self.state),
                 page_indptr=full(n + 1), page_indices=full(page_capacity), last_page_len=full(n),
                 qo_indptr=full(n + 1), slot_map=full(token_capacity, torch.int64),
                 positions=full(token_capacity))
        d["kv_len_out"] = d["kv_len"] if in_place else full(len(self.kv_len))
        d["ring_state_out"] = d["ring_state"] if in_place else full(2)
        if workspace is None:
            workspace = torch.zeros(256, dtype=torch.uint8, device="cuda")
        d["workspace"] = workspace
        B.fi_page_table_step(n, None if null_slots else d["slots"], d["new_len"], len(self.kv_len),
                             self.max_pages, self.P, d["kv_len"], d["kv_len_out"],
                             d["block_table"], d["free_ring"], len(self.ring), d["ring_state"],
                             d["ring_state_out"], d["page_indptr"],
                             d["page_indices"] if page_capacity else None, page_capacity,
                             d["last_page_len"], d["qo_indptr"],
                             d["slot_map"] if token_capacity else None,
                             d["positions"] if positions else None, token_capacity, workspace)
        d["status"] = B.fi_check_device_status(workspace)
        return {k: (v.cpu().numpy() if hasattr(v, "cpu") else v) for k, v in d.items()}

    def want(self, slots, new_len, page_capacity, token_capacity):
        return _step.page_table_step(slots, new_len, self.kv_len, self.table, self.ring,
                                     self.state, self.P, page_capacity, token_capacity)

    def take(self, w):
        self.kv_len[:], self.table[:], self.ring[:] = w["kv_len"], w["block_table"], w["free_ring"]
        self.state[:] = w["ring_state"]


def _check(got, want, slots, page_capacity, in_place, positions=True):
    assert got["status"] == B.FI_OK
    n = len(want["page_indices"])
    for k in ("page_indptr", "last_page_len", "qo_indptr", "block_table", "free_ring"):
        assert np.array_equal(got[k], want[k]), k
    assert np.array_equal(got["page_indices"][:n], want["page_indices"])
    assert np.all(got["page_indices"][n:] == -77)          # behind the last one: as it was
    cap = len(want["slot_map"])
    assert np.array_equal(got["slot_map"][:cap], want["slot_map"])
    assert np.array_equal(got["positions"][:cap], want["positions"] if positions
                          else np.full(cap, -77))
    assert np.array_equal(got["ring_state_out"], want["ring_state"])
    if in_place:
        assert np.array_equal(got["kv_len_out"], want["kv_len"])
    else:
        named = sorted(s for s in slots if s >= 0)
        rest = np.setdiff1d(np.arange(len(want["kv_len"])), named)
        assert np.array_equal(got["kv_len_out"][named], want["kv_len"][named])
        assert np.all(got["kv_len_out"][rest] == -77)


@pytest.mark.parametrize("P", [1, 16, 32, 48])
@pytest.mark.parametrize("batch,slots,kv,new", [(1, 1, 0, 1), (1, 5, 100, 40), (7, 9, 33, 1),
                                                (33, 40, 200, 20), (300, 300, 50, 3),
                                                (1500, 1600, 40, 2)])
def test_steps_of_many_shapes(P, batch, slots, kv, new):
    rng = np.random.default_rng(batch * 100 + P)
    s = Server(slots, -(-(kv + 4 * new + 8) // P) + 1, P, slots * (-(-(kv + 4 * new + 8) // P) + 1), P)
    s.fill(rng.integers(0, kv + 1, slots))
    for i in range(3):
        order = rng.permutation(slots)[:batch]
        order = np.where(rng.random(batch) < 0.15, -1 - i, order)
        add = np.array([rng.integers(-min(s.kv_len[x], 30), new + 1) if x >= 0 else 9 for x in order])
        caps = (int(s.kv_len.sum()) // P + slots + batch * new + 5, batch * new + 3 * i)
        want = s.want(order, add, *caps)
        got = s.step(order, add, *caps, in_place=bool(i % 2), positions=i != 1)
        _check(got, want, order, caps[0], bool(i % 2), positions=i != 1)
        s.take(want)


def test_a_long_run_of_steps_keeps_every_page_once():
    """Requests grow, shrink and end over 60 steps around a small ring: no page
    is ever held twice, none is lost."""
    rng = np.random.default_rng(3)
    s = Server(12, 8, 16, 60, 4)
    torch = _torch()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for i in range(60):
        order = rng.permutation(12)[:rng.integers(1, 13)]
        add = np.array([-s.kv_len[x] if rng.random() < 0.15 else
                        min(rng.integers(-min(5, s.kv_len[x]), 30), 128 - s.kv_len[x])
                        for x in order])
        try:
            want = s.want(order, add, 100, 400)
        except _step.StepError:
            got = s.step(order, add, 100, 400, workspace=ws)
            assert got["status"] == B.FI_ERR_OUT_OF_PAGES
            assert np.array_equal(got["kv_len"], s.kv_len)
            continue
        got = s.step(order, add, 100, 400, workspace=ws)
        _check(got, want, order, 100, True)
        s.take(want)
        held = [p for x in range(12) for p in s.table[x, :-(-s.kv_len[x] // 16)]]
        free = [s.ring[(s.state[0] + j) % 60] for j in range(s.state[1])]
        assert sorted(held + free) == list(range(60))


def test_slots_may_be_left_out():
    s = Server(5, 6, 16, 30, 1)
    s.fill([3, 0, 16, 31, 17])
    want = s.want([0, 1, 2, 3, 4], [1, 5, 1, -31, 2], 40, 9)
    got = s.step([0, 1, 2, 3, 4], [1, 5, 1, -31, 2], 40, 9, null_slots=True)
    _check(got, want, [0, 1, 2, 3, 4], 40, True)


def test_largest_batch_and_slots():
    s = Server(262144, 2, 16, 20000, 2)
    rng = np.random.default_rng(8)
    order = rng.permutation(262144)[:8192]
    s.fill([0])
    add = rng.integers(0, 33, 8192)
    want = s.want(order, add, 20000, 8192 * 32)
    _check(s.step(order, add, 20000, 8192 * 32), want, order, 20000, True)


@pytest.mark.parametrize("capacity", [8192, 16384])
def test_largest_batch_with_few_new_rows(capacity):
    """(few output entries: the blocks are one cluster)"""
    s = Server(262144, 2, 16, 20000, 4)
    rng = np.random.default_rng(10)
    order = rng.permutation(262144)[:8192]
    s.fill([0])
    add = rng.integers(0, 2, 8192)
    want = s.want(order, add, capacity, capacity)
    _check(s.step(order, add, capacity, capacity), want, order, capacity, True)


@pytest.mark.parametrize("what,status", [
    ("pages", B.FI_ERR_OUT_OF_PAGES), ("row", B.FI_ERR_OUT_OF_PAGES),
    ("page_capacity", B.FI_ERR_OUT_OF_PAGES), ("token_capacity", B.FI_ERR_OUT_OF_PAGES),
    ("twice", B.FI_ERR_DEVICE_BOUNDS), ("slot", B.FI_ERR_DEVICE_BOUNDS),
    ("drop", B.FI_ERR_DEVICE_BOUNDS), ("negative", B.FI_ERR_DEVICE_BOUNDS),
    ("head", B.FI_ERR_DEVICE_BOUNDS), ("count", B.FI_ERR_DEVICE_BOUNDS),
    ("full_ring", B.FI_ERR_DEVICE_BOUNDS), ("huge", B.FI_ERR_DEVICE_BOUNDS)])
def test_a_step_that_cannot_be_made_changes_nothing(what, status):
    s = Server(4, 5, 16, 20, 1)
    s.fill([10, 20, 30, 0])
    slots, add, caps = [2, 0, 3], [5, 5, 5], [30, 15]
    if what == "pages":
        s.state[1] = 1
    elif what == "row":
        add[2] = 81
        caps[1] = 200
    elif what == "page_capacity":
        caps[0] = 4
    elif what == "token_capacity":
        caps[1] = 14
    elif what == "twice":
        slots[2] = 2
    elif what == "slot":
        slots[1] = 4
    elif what == "drop":
        add[0] = -31
    elif what == "negative":
        s.kv_len[0] = -1
    elif what == "head":
        s.state[0] = 20
    elif what == "count":
        s.state[1] = 21
    elif what == "full_ring":
        s.state[1] = 20
        add[0] = -30
    elif what == "huge":
        add[0] = 2 ** 31 - 1
    for in_place in (True, False):
        got = s.step(slots, add, *caps, in_place=in_place)
        assert got["status"] == status
        assert np.array_equal(got["block_table"], s.table)
        assert np.array_equal(got["free_ring"], s.ring)
        assert np.array_equal(got["ring_state_out"], s.state)
        for x in slots:
            if x < 4:
                assert got["kv_len_out"][x] == s.kv_len[x]
        assert not got["page_indptr"].any() and not got["qo_indptr"].any()
        assert not got["last_page_len"].any()
        assert np.all(got["slot_map"] == -1) and not got["positions"].any()
        assert np.all(got["page_indices"] == -77)


def test_captured_steps_advance_the_requests():
    """The step captured once and replayed: each replay is a further step."""
    torch = _torch()
    P, n = 16, 6
    s = Server(n, 20, P, 100, 5)
    s.fill([1, 16, 40, 0, 5, 31])
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    kv, table, ring, state = dev(s.kv_len), dev(s.table), dev(s.ring), dev(s.state)
    new, slots = dev([1] * n), dev(range(n))
    i32 = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")
    indptr, indices, last, qo, pos = i32(n + 1), i32(80), i32(n), i32(n + 1), i32(200)
    smap = torch.zeros(200, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.fi_page_table_step(n, slots, new, n, 20, P, kv, kv, table, ring, 100, state, state,
                             indptr, indices, 80, last, qo, smap, pos, 200, ws)
    for i in range(20):
        add = np.random.default_rng(i).integers(-2, 5, n).clip(-s.kv_len)
        want = s.want(list(range(n)), add, 80, 200)
        new.copy_(dev(add))
        g.replay()
        assert B.fi_check_device_status(ws) == B.FI_OK
        assert np.array_equal(kv.cpu().numpy(), want["kv_len"])
        assert np.array_equal(table.cpu().numpy(), want["block_table"])
        assert np.array_equal(ring.cpu().numpy(), want["free_ring"])
        assert np.array_equal(smap.cpu().numpy(), want["slot_map"])
        assert np.array_equal(indptr.cpu().numpy(), want["page_indptr"])
        s.take(want)


# ---- append ----------------------------------------------------------------------------------
def _values(rng, shape, dtype):
    """Random values of unequal rows as a tensor of dtype, and in float64."""
    torch = _torch()
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, shape[:-1] + (1,)))
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float16)
    return t, t.double().numpy()


def _append(kn, vn, smap, kc, vc, ks, vs, dtype, kv_dtype, layout, P, stride=0, pages=None,
            page_stride=0):
    """The call on device copies; caches come and go as [page][slot][head][dim]."""
    torch = _torch()
    H, d = kn.shape[1], kn.shape[2]
    lay = (lambda a: a) if layout == "NHD" else (lambda a: a.transpose(1, 2))
    dev = lambda a: (a if torch.is_tensor(a) else torch.from_numpy(a)).cuda()
    k, v = [lay(dev(c)).contiguous() for c in (kc, vc)]
    kst, vst = [None if a is None else dev(a.astype(np.float32)) for a in (ks, vs)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.fi_append_paged_kv(len(smap), dev(np.asarray(smap, dtype=np.int64)), dev(kn), dev(vn), stride,
                         B.FI_DTYPE_BF16 if dtype == "bf16" else B.FI_DTYPE_FP16, H, d, k, v,
                         kv_dtype, B.LAYOUTS[layout], page_stride, pages or kc.shape[0], P, kst, vst, ws)
    st = B.fi_check_device_status(ws)
    back = [lay(c).cpu() for c in (k, v)]
    return back + [None if a is None else a.cpu().numpy().astype(np.float64) for a in (kst, vst)] + [st]


def _runs(rng, n_pages, P, kind):
    """A slot map of whole and part pages in a random order of pages."""
    out = []
    for page in rng.permutation(n_pages):
        first = int(rng.integers(0, P)) if rng.random() < 0.6 else 0
        n = {"one": 1, "full": P - first, "some": int(rng.integers(1, P - first + 1))}[kind]
        out += [int(page) * P + first + i for i in range(n)]
        if rng.random() < 0.3:
            out.append(-1 - int(rng.integers(0, 3)))
    return out


@pytest.mark.parametrize("kind", ["one", "some", "full"])
@pytest.mark.parametrize("layout,dtype", [("NHD", "bf16"), ("HND", "fp16")])
@pytest.mark.parametrize("d,P,H", [(64, 16, 3), (64, 32, 8), (128, 16, 8), (128, 32, 1), (256, 16, 2),
                                   (256, 32, 5)])
def test_quantising_append(d, P, H, layout, dtype, kind):
    rng = np.random.default_rng(d + P + H)
    n_pages = 37
    smap = _runs(rng, n_pages, P, kind)
    kn, k64 = _values(rng, (len(smap), H, d), dtype)
    vn, v64 = _values(rng, (len(smap), H, d), dtype)
    kc, vc = [rng.integers(0, 127, (n_pages, P, H, d)).astype(np.uint8) |
              (rng.integers(0, 2, (n_pages, P, H, d)).astype(np.uint8) << 7) for _ in range(2)]
    ks, vs = [np.exp2(rng.integers(-14, 0, (n_pages, H))).astype(np.float64) for _ in range(2)]
    k, v, ks2, vs2, st = _append(kn, vn, smap, kc, vc, ks, vs, dtype, B.FI_DTYPE_E4M3_PAGE, layout, P)
    assert st == B.FI_OK
    for x, c, s, got, gs in ((k64, kc, ks, k, ks2), (v64, vc, vs, v, vs2)):
        want, ws = _step.append_page_scaled(smap, x, c, s, P)
        assert np.array_equal(gs, ws)
        assert np.array_equal(got.numpy(), want)


def test_append_special_values():
    """Zeros, NaN, infinities, the largest and the smallest values; an older
    row whose code is NaN; a scale that is no power of two."""
    torch = _torch()
    P, H, d = 16, 2, 64
    x = np.zeros((8, H, d))
    x[1, 0, 3], x[2, 0, 5], x[2, 1, 0] = np.nan, np.inf, -np.inf
    x[3, :, 7] = 3.0e38
    x[4, :, 9] = 2.0 ** -130
    x[5], x[6], x[7] = 448.0, 0.1, -7.0
    smap = [0, 16, 17, 32, 48, 64, 85, 103]           # pages 5 and 6 keep older rows
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    x64 = t.double().numpy()
    kc = np.full((7, P, H, d), 0x35, dtype=np.uint8)
    kc[5, 2, 0, 0] = 0x7f
    ks = np.full((7, H), 2.0 ** -14)
    ks[6] = np.float64(np.float32(0.3))
    k, _, ks2, _, st = _append(t, t, smap, kc, kc, ks, ks, "bf16", B.FI_DTYPE_E4M3_PAGE, "NHD", P)
    assert st == B.FI_OK
    want, ws = _step.append_page_scaled(smap, x64, kc, ks, P)
    assert np.array_equal(ks2, ws)
    got = _step.e4m3_value(k.numpy())
    assert np.array_equal(got, _step.e4m3_value(want), equal_nan=True)
    assert np.isnan(got[1, 0, 0, 3]) and np.isnan(got[1, 1, 0, 5]) and np.isnan(got[5, 2, 0, 0])
    assert ws[3, 0] == 2.0 ** -100 and ws[0, 0] == 2.0 ** -100   # the tiny row, the zero row


def test_append_row_and_page_strides():
    """k and v as parts of a fused projection's rows; K and V pages of one buffer."""
    torch = _torch()
    rng = np.random.default_rng(9)
    P, H, d, T = 16, 4, 128, 40
    rows, r64 = _values(rng, (T, 4 * H, d), "bf16")
    smap = np.arange(5, 5 + T)
    kv = torch.zeros(6, 2, P, H, d, dtype=torch.uint8, device="cuda")
    ks = torch.full((6, H), 2.0 ** -100, device="cuda")
    vs = ks.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    r = rows.cuda()
    B.fi_append_paged_kv(T, torch.from_numpy(smap).cuda(), r[:, 2 * H:3 * H], r[:, 3 * H:],
                         4 * H * d, B.FI_DTYPE_BF16, H, d, kv, kv[:, 1], B.FI_DTYPE_E4M3_PAGE,
                         B.FI_LAYOUT_NHD, 2 * P * H * d, 6, P, ks, vs, ws)
    assert B.fi_check_device_status(ws) == B.FI_OK
    zero = np.zeros((6, P, H, d), dtype=np.uint8)
    for i, part in ((0, r64[:, 2 * H:3 * H]), (1, r64[:, 3 * H:])):
        want, s = _step.append_page_scaled(smap, part, zero, np.full((6, H), 2.0 ** -100), P)
        assert np.array_equal(kv[:, i].cpu().numpy(), want)
        assert np.array_equal((ks, vs)[i].cpu().numpy(), s)


@pytest.mark.parametrize("layout,dtype", [("NHD", "bf16"), ("HND", "fp16")])
@pytest.mark.parametrize("d,P,H", [(64, 16, 3), (128, 32, 8), (256, 16, 2)])
def test_append_to_a_16_bit_cache(d, P, H, layout, dtype):
    torch = _torch()
    rng = np.random.default_rng(d)
    smap = _runs(rng, 30, P, "some")
    kn, _ = _values(rng, (len(smap), H, d), dtype)
    vn, _ = _values(rng, (len(smap), H, d), dtype)
    kc = torch.full((30, P, H, d), 3.0, dtype=kn.dtype)
    k, v, _, _, st = _append(kn, vn, smap, kc, kc, None, None, dtype,
                             B.FI_DTYPE_BF16 if dtype == "bf16" else B.FI_DTYPE_FP16, layout, P)
    assert st == B.FI_OK
    for rows, got in ((kn, k), (vn, v)):
        want = kc.clone()
        for t, s in enumerate(smap):
            if s >= 0:
                want[s // P, s % P] = rows[t]
        assert torch.equal(got, want)


@pytest.mark.parametrize("kv", ["page", "same"])
def test_append_skips_and_reports_slots_outside_the_cache(kv):
    torch = _torch()
    rng = np.random.default_rng(1)
    P, H, d = 16, 2, 64
    smap = [3, 4, 8 * P - 1, 8 * P, 9 * P + 3, 2 ** 40, -1, 20]   # pages 8, 9 and further: none
    kn, k64 = _values(rng, (len(smap), H, d), "bf16")
    if kv == "page":
        kc = np.zeros((12, P, H, d), dtype=np.uint8)              # the call is told of 8 pages
        ks = np.full((12, H), 2.0 ** -100)
        k, _, ks2, _, st = _append(kn, kn, smap, kc, kc, ks, ks, "bf16", B.FI_DTYPE_E4M3_PAGE,
                                   "NHD", P, pages=8)
        want, ws = _step.append_page_scaled([s if s < 8 * P else -1 for s in smap], k64, kc, ks, P)
        assert np.array_equal(k.numpy(), want) and np.array_equal(ks2, ws)
    else:
        kc = torch.zeros(12, P, H, d, dtype=torch.bfloat16)
        k, _, _, _, st = _append(kn, kn, smap, kc, kc, None, None, "bf16", B.FI_DTYPE_BF16, "NHD",
                                 P, pages=8)
        want = kc.clone()
        for t in (0, 1, 2, 7):
            want[smap[t] // P, smap[t] % P] = kn[t]
        assert torch.equal(k, want)
    assert st == B.FI_ERR_DEVICE_BOUNDS
