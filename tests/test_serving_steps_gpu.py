"""The operators as a server runs them, one step after the other: the page
table of the step from the device's lengths, the step's K and V quantised into
the slots it names, attention over the cache with the step's own table. Prompts
in chunks, decode rows, rejected draft tokens, requests that end and slots that
are used again; every step's table, cache, scales and outputs are compared with
plain implementations."""
import numpy as np
import pytest

from paged_kv_attention_27_gb300 import binding as B

from . import _page8, _step
from ._gpu import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()
    return B.lib()


class PlainCache:
    """The float64 side: lengths, pages, codes and scales."""

    def __init__(self, slots, max_pages, P, hkv, d, pool, seed):
        rng = np.random.default_rng(seed)
        self.P = P
        self.kv_len = np.zeros(slots, dtype=np.int32)
        self.table = np.full((slots, max_pages), -1, dtype=np.int32)
        self.ring = rng.permutation(pool).astype(np.int32)
        self.state = np.array([0, pool], dtype=np.int32)
        self.codes = [rng.integers(0, 256, (pool, P, hkv, d)).astype(np.uint8) for _ in range(2)]
        self.scale = [np.full((pool, hkv), 3.0) for _ in range(2)]   # stale: never used

    def step(self, slots, new, caps):
        r = _step.page_table_step(slots, new, self.kv_len, self.table, self.ring, self.state, self.P,
                                  *caps)
        self.kv_len[:], self.table[:], self.ring[:] = r["kv_len"], r["block_table"], r["free_ring"]
        self.state[:] = r["ring_state"]
        return r


def _batch(plain, r, slots, qo, q, hq, hkv, d, dtype, layout, window):
    """The step as a _page8.Batch (for its plan, reference and comparison)."""
    b = _page8.Batch([1], hq, hkv, d, plain.P, layout, dtype, seed=0)
    b.kv_lens = [int(plain.kv_len[s]) if s >= 0 else 0 for s in slots]
    b.qo_lens, b.decode, b.causal, b.window = list(qo), False, True, window
    b.page_indptr, b.page_indices = r["page_indptr"].astype(np.int32), r["page_indices"].astype(np.int32)
    b.last_page_len, b.qo_indptr = r["last_page_len"].astype(np.int32), r["qo_indptr"].astype(np.int32)
    b.num_pages, b.rows, b.q = len(plain.ring), int(sum(qo)), q
    b.codes, b.scale = plain.codes, plain.scale
    return b


@pytest.mark.parametrize("hq,hkv,d,P,layout,dtype,window", [
    (8, 2, 128, 16, "NHD", "bf16", -1), (8, 1, 64, 32, "HND", "fp16", -1),
    (2, 2, 256, 16, "HND", "bf16", 50)])
def test_serving_steps(hq, hkv, d, P, layout, dtype, window):
    import torch
    rng = np.random.default_rng(d)
    slots_n, max_pages, pool, T = 6, -(-400 // P), 4 * -(-400 // P), 160
    plain = PlainCache(slots_n, max_pages, P, hkv, d, pool, 1)
    dev = lambda a, t=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    kv_len, table, ring, state = (dev(plain.kv_len), dev(plain.table), dev(plain.ring),
                                  dev(plain.state))
    lay = (lambda a: a) if layout == "NHD" else (lambda a: a.transpose(1, 2).contiguous())
    k, v = [lay(torch.from_numpy(c).cuda()).clone() for c in plain.codes]
    ks, vs = [torch.from_numpy(s.astype(np.float32)).cuda() for s in plain.scale]
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    n = 5
    slots, new = i32(n), i32(n)
    indptr, indices, last, qo, pos = i32(n + 1), i32(pool), i32(n), i32(n + 1), i32(T)
    smap = torch.zeros(T, dtype=torch.int64, device="cuda")
    ws = torch.zeros(B.FI_STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    # the projections' output of a padded batch of T rows: q, k and v of a row
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    rows = torch.zeros(T, hq + 2 * hkv, d, dtype=dt, device="cuda")
    fi_dt = B.FI_DTYPE_BF16 if dtype == "bf16" else B.FI_DTYPE_FP16

    def prepare():
        B.fi_page_table_step(n, slots, new, slots_n, max_pages, P, kv_len, kv_len, table, ring, pool,
                             state, state, indptr, indices, pool, last, qo, smap, pos, T, ws)
        B.fi_append_paged_kv(T, smap, rows[:, hq:hq + hkv], rows[:, hq + hkv:], rows.stride(0),
                             fi_dt, hkv, d, k, v, B.FI_DTYPE_E4M3_PAGE, B.LAYOUTS[layout], 0, pool, P,
                             ks, vs, ws)

    graph = torch.cuda.CUDAGraph()      # the preparation, captured once
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        prepare()
    for step in range(24):
        order = [int(s) for s in rng.permutation(slots_n)[:n]]
        if step % 5 == 4:
            order[rng.integers(n)] = -1                      # a padded row
        add = []
        for s in order:
            have = int(plain.kv_len[s]) if s >= 0 else 0
            if have == 0:
                add.append(int(rng.integers(1, 90)))         # a prompt
            elif have > 300 or rng.random() < 0.1:
                add.append(-have)                            # it ends
            elif rng.random() < 0.15:
                add.append(-int(rng.integers(1, min(have, 6) + 1)))   # rejected drafts
            else:
                add.append(int(rng.choice([1, 1, 1, 4, 30])))
        while sum(max(x, 0) for x, s in zip(add, order) if s >= 0) > T:
            add[int(np.argmax(add))] = 1
        try:
            r = plain.step(order, add, (pool, T))
        except _step.StepError:
            continue                                          # a full pool: tested elsewhere
        real = [max(x, 0) if s >= 0 else 0 for x, s in zip(add, order)]
        x = rng.standard_normal((T, hq + 2 * hkv, d)) * np.exp2(rng.integers(-3, 4, (T, 1, 1)))
        rows.copy_(torch.from_numpy(x).to(dt))
        slots.copy_(dev(order))
        new.copy_(dev(add))
        if step % 3:
            prepare()
        else:
            graph.replay()
        assert B.fi_check_device_status(ws) == B.FI_OK
        got = rows.double().cpu().numpy()
        for i, part in ((0, got[:, hq:hq + hkv]), (1, got[:, hq + hkv:])):
            plain.codes[i], plain.scale[i] = _step.append_page_scaled(
                r["slot_map"], part, plain.codes[i], plain.scale[i], P)
        assert np.array_equal(kv_len.cpu().numpy(), plain.kv_len)
        assert np.array_equal(smap.cpu().numpy(), r["slot_map"])
        assert np.array_equal(pos.cpu().numpy(), r["positions"])
        for t, c in ((k, plain.codes[0]), (v, plain.codes[1])):
            assert np.array_equal(lay(t).cpu().numpy() if layout == "NHD"
                                  else t.transpose(1, 2).cpu().numpy(), c)
        for t, s in ((ks, plain.scale[0]), (vs, plain.scale[1])):
            assert np.array_equal(t.cpu().numpy().astype(np.float64), s)
        m = sum(real)
        if m == 0:
            continue
        # the plan from the lengths, which the server knows; the page table from the device
        b = _batch(plain, r, order, real, rows[:m, :hq].cpu(), hq, hkv, d, dtype, layout, window)
        plan = b.plan(B, num_sms=torch.cuda.get_device_properties(0).multi_processor_count)
        run_ws = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
        q = rows[:m, :hq].contiguous()
        out = torch.empty(m, hq, d, dtype=dt, device="cuda")
        lse = torch.empty(m, hq, dtype=torch.float32, device="cuda")
        B.fi_batch_prefill_paged(plan, q, qo, k, v, B.LAYOUTS[layout], 0, pool, indptr, indices, last,
                                 b.sm_scale, 1.0, 1.0, out, lse, run_ws, k_head_scale=ks, v_head_scale=vs)
        assert B.fi_check_device_status(run_ws) == B.FI_OK
        _page8.compare(b, out, lse, _page8.reference(b), what=f"step {step}")
