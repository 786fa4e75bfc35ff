"""Cases of the operators around a paged KV cache held in 8 bits.

A serving step over such a cache has three parts, and each is an operator here:

* ``table``: the requests' lengths advance on the device; pages are taken from (or returned to) a
  ring of free pages, and the step's page table, row offsets and slot map are built from them;
* ``append``: the step's new K and V rows are quantised to FP8 E4M3 and stored in their slots. Every
  (page, kv head) has one scale, a power of two, which only grows while the page fills;
* ``decode`` / ``prefill``: attention of one query row, or of a chunk of rows, per request over that
  cache with its scales.

``run`` computes them in their plain form (elementary tensor operations in 32 bits), or, where
``own`` is true, by the library's calls.
"""
import math
import random

import torch

own = False

INT = torch.int32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MIN_EXP = -100   # the smallest scale is 2^-100 (a page of zeros)


def listed():
    return [
        # one decode step of a server with 256 running requests
        dict(name="table_decode", op="table", batch=256, max_requests=512, kv_lo=16, kv_hi=8192,
             new_lo=1, new_hi=1, drop=0.0, pad=0.0, page=16, lens=1),
        # a full step of a large server: chunks, decode rows, rejected draft tokens, a padded batch
        dict(name="table_mixed", op="table", batch=1536, max_requests=2048, kv_lo=1, kv_hi=8192,
             new_lo=1, new_hi=64, drop=0.1, pad=0.05, page=16, lens=2),
        # the new rows of one decode step of 128 requests
        dict(name="append_decode", op="append", batch=128, kv_lo=16, kv_hi=4096, q_lo=1, q_hi=1,
             hkv=8, d=128, page=16, layout="NHD", dtype="bf16", fused=True, lens=3),
        # prompts of up to 4K tokens
        dict(name="append_prompts", op="append", batch=8, kv_lo=0, kv_hi=0, q_lo=1000, q_hi=4096,
             hkv=8, d=128, page=16, layout="NHD", dtype="bf16", fused=True, lens=4),
        # ragged chunks behind existing tokens, wide heads, the other layout and type
        dict(name="append_chunks_d256", op="append", batch=24, kv_lo=1, kv_hi=2000, q_lo=1,
             q_hi=150, hkv=4, d=256, page=32, layout="HND", dtype="fp16", fused=False, lens=5),
        # the smallest attention call: a handful of short requests
        dict(name="decode_small", op="decode", batch=4, kv_lo=1, kv_hi=100, hq=8, hkv=2, d=64,
             page=16, layout="NHD", dtype="bf16", window=-1, lens=6),
        # 64 requests with one kv head per query head
        dict(name="decode_mha", op="decode", batch=64, kv_lo=512, kv_hi=4096, hq=32, hkv=32, d=128,
             page=16, layout="NHD", dtype="bf16", window=-1, lens=7),
        # 128 requests with eight query heads per kv head, lengths from short to long
        dict(name="decode_gqa", op="decode", batch=128, kv_lo=128, kv_hi=16384, hq=64, hkv=8, d=128,
             page=16, layout="HND", dtype="bf16", window=-1, lens=8),
        # wide heads in fp16 with a sliding window
        dict(name="decode_d256_window", op="decode", batch=56, kv_lo=700, kv_hi=16384, hq=16, hkv=8,
             d=256, page=32, layout="NHD", dtype="fp16", window=4095, lens=9),
        # a draft's rows checked against the cache: a few rows per request
        dict(name="prefill_verify", op="prefill", batch=48, kv_lo=300, kv_hi=8192, q_lo=1, q_hi=9,
             hq=32, hkv=8, d=128, page=16, layout="NHD", dtype="bf16", window=-1, lens=10),
        # chunks of a long prompt
        dict(name="prefill_long_chunk", op="prefill", batch=2, kv_lo=20000, kv_hi=32000, q_lo=400,
             q_hi=512, hq=64, hkv=8, d=128, page=16, layout="NHD", dtype="bf16", window=-1, lens=11),
        # whole prompts
        dict(name="prefill_prompts", op="prefill", batch=4, kv_lo=0, kv_hi=0, q_lo=3300, q_hi=4096,
             hq=64, hkv=8, d=128, page=16, layout="NHD", dtype="bf16", window=-1, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "decode", "prefill"])
    case = dict(op=op, page=rng.choice([16, 32]), lens=rng.randrange(1 << 20))
    if op == "table":
        batch = _log(rng, 1, 1536)
        lo = _log(rng, 1, 1000)
        case.update(batch=batch, max_requests=batch + rng.randrange(600), kv_lo=lo,
                    kv_hi=_log(rng, lo, 8192), new_lo=1, new_hi=_log(rng, 1, 64),
                    drop=rng.choice([0.0, 0.1, 0.5]), pad=rng.choice([0.0, 0.1]))
        return case
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8, 16, 32] if d < 256 else [1, 2, 4, 8])
    case.update(d=d, hkv=hkv, layout=rng.choice(["NHD", "HND"]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "append":
        batch = _log(rng, 1, 256)
        most = max(1, min(4096, 8_000_000 // (batch * hkv * d)))
        q_hi = _log(rng, 1, most)
        case.update(batch=batch, kv_lo=0, kv_hi=_log(rng, 1, 500), q_lo=max(1, q_hi // 4), q_hi=q_hi,
                    fused=rng.random() < 0.5)
        return case
    g = rng.choice([1, 2, 4, 8])
    window = rng.choice([-1, -1, rng.randrange(1, 2000)])
    if op == "decode":
        batch = _log(rng, 1, 128)
        most = max(64, min(32768, 500_000_000 // (batch * hkv * d)))
        hi = _log(rng, 32, most)
        case.update(batch=batch, hq=g * hkv, kv_lo=max(1, hi // rng.choice([2, 10, 100])), kv_hi=hi,
                    window=window)
        return case
    batch = _log(rng, 1, 64)
    q_hi = _log(rng, 2, max(2, min(2048, 8192 // batch)))
    most = max(1, min(32768, 1_000_000_000 // (batch * g * hkv * q_hi),
                      500_000_000 // (batch * hkv * d)))
    hi = _log(rng, 1, most)
    case.update(batch=batch, hq=g * hkv, q_lo=max(1, q_hi // 3), q_hi=q_hi, kv_lo=hi // 4, kv_hi=hi,
                window=window)
    return case


# ---- sizes and inputs ---------------------------------------------------------------------------
def _lens(case):
    """Per request: (keys before this call, rows of this call). Lengths are spread over their
    logarithm; the first request has the longest of each."""
    rng = random.Random(case["lens"])
    n = case["batch"]
    ctx = [0 if case["kv_hi"] == 0 else
           int(round(math.exp(rng.uniform(math.log(max(case["kv_lo"], 1)),
                                          math.log(max(case["kv_hi"], 1)))))) for _ in range(n)]
    ctx[0] = case["kv_hi"]
    if case["op"] == "decode":
        return [c - 1 for c in ctx], [1] * n
    if case["op"] == "table":
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        for b in range(n):
            if rng.random() < case["drop"]:
                new[b] = -rng.randint(1, min(ctx[b], 40))
        return ctx, new
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    q[0] = case["q_hi"]
    return ctx, q


def _indptr(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s (at least 2^MIN_EXP), for amax >= 0."""
    frac, exp = torch.frexp(amax)
    exp = torch.where(frac <= 0.875, exp - 9, exp - 8)
    exp = torch.where(amax > 0, exp, MIN_EXP).clamp(min=MIN_EXP).to(INT)
    return ((exp + 127) << 23).view(torch.float32)


def _quantised(x):
    """A cache of real values [page][slot][head][dim] as E4M3 codes and page scales [page][head]."""
    s = _scale_of(x.abs().amax(dim=(1, 3)))
    codes = (x / s[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), s


def _laid(x, layout):
    return x.contiguous() if layout == "NHD" else x.transpose(1, 2).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = dict(device="cuda")
    P = case["page"]
    ctx, new = _lens(case)

    def ints(x, dtype=INT):
        return torch.tensor(x, dtype=dtype, **dev)

    if case["op"] == "table":
        n, slots_n = case["batch"], case["max_requests"]
        rng = random.Random(case["lens"] + 1)
        live = [rng.random() >= case["pad"] for _ in range(n)]
        live[0] = True
        slots = torch.randperm(slots_n, generator=gen, **dev)[:n].to(INT)
        slots = torch.where(ints(live, torch.bool), slots, -1)
        held = [-(-c // P) if ok else 0 for c, ok in zip(ctx, live)]
        width = -(-(max(ctx) + 64 + P) // P)
        grow = [max(x, 0) if ok else 0 for x, ok in zip(new, live)]
        pages_after = sum(-(-(c + x) // P) for c, x, ok in zip(ctx, new, live) if ok)
        ids = torch.randperm(sum(held) + sum(grow) // P + 2 * n + 100, generator=gen, **dev).to(INT)
        table = torch.full((slots_n, width), -1, dtype=INT, **dev)
        row = torch.repeat_interleave(torch.arange(n, **dev), ints(held, torch.int64))
        col = torch.arange(sum(held), **dev) - ints(_indptr(held)[:-1], torch.int64)[row]
        table[slots[row].long(), col] = ids[:sum(held)]
        kv_len = torch.zeros(slots_n, dtype=INT, **dev)
        keep = ints(live, torch.bool)
        kv_len[slots[keep].long()] = ints(ctx)[keep]
        cap = ids.numel()
        head = int(seed) % cap
        free = ids[sum(held):]
        ring = torch.full((cap,), -1, dtype=INT, **dev)
        ring[(head + torch.arange(free.numel(), **dev)) % cap] = free
        page_cap, tok_cap = pages_after + 64, sum(grow) + 16

        def blank(m, dtype=INT, value=-1):
            return torch.full((m,), value, dtype=dtype, **dev)

        return dict(case=case, slots=slots, new_len=ints(new), kv_len=kv_len, table=table, ring=ring,
                    ring_state=ints([head, free.numel()]), kv_len_out=blank(slots_n),
                    ring_state_out=blank(2), page_indptr=blank(n + 1), page_indices=blank(page_cap),
                    last_page_len=blank(n), qo_indptr=blank(n + 1),
                    slot_map=blank(tok_cap, torch.int64), positions=blank(tok_cap),
                    workspace=torch.zeros(256, dtype=torch.uint8, **dev))

    total = [c + x for c, x in zip(ctx, new)]
    pages = [-(-t // P) for t in total]
    indptr, qo = _indptr(pages), _indptr(new)
    num_pages = indptr[-1] + 7
    indices = torch.randperm(num_pages, generator=gen, **dev)[:indptr[-1]].to(INT)
    hkv, d, dt = case["hkv"], case["d"], TYPES[case["dtype"]]
    T = qo[-1]
    # keys have channels of unequal size; values are plain
    chan = torch.exp(0.5 * torch.randn(hkv, d, generator=gen, **dev))
    page_indptr, qo_indptr = ints(indptr), ints(qo)
    last = ints([(t - 1) % P + 1 if t else 0 for t in total])

    def values(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float32, **dev)

    k_codes, k_scale = _quantised(values(num_pages, P, hkv, d) * chan)
    v_codes, v_scale = _quantised(values(num_pages, P, hkv, d))
    st = dict(case=case, k=_laid(k_codes, case["layout"]), v=_laid(v_codes, case["layout"]),
              k_scale=k_scale, v_scale=v_scale, page_indptr=page_indptr, page_indices=indices,
              last_page_len=last, qo_indptr=qo_indptr, num_pages=num_pages)
    if case["op"] == "append":
        # the new rows' slots, as the page table step gives them
        req = torch.repeat_interleave(torch.arange(case["batch"], **dev), ints(new, torch.int64))
        pos = torch.arange(T, **dev) - ints(qo[:-1], torch.int64)[req] + ints(ctx, torch.int64)[req]
        page = indices.long()[ints(indptr[:-1], torch.int64)[req] + pos // P]
        # k and v of a fused projection's output (with twice as many query heads), or separate
        hq = 2 * hkv if case["fused"] else 0
        rows = torch.empty(T, (hq + 2 * hkv) * d, dtype=dt, **dev)
        rows[:, hq * d:(hq + hkv) * d] = (values(T, hkv, d) * chan).reshape(T, -1).to(dt)
        rows[:, (hq + hkv) * d:] = values(T, hkv * d).to(dt)
        k_new, v_new = rows[:, hq * d:(hq + hkv) * d], rows[:, (hq + hkv) * d:]
        if not case["fused"]:
            k_new, v_new = k_new.contiguous(), v_new.contiguous()
        st.update(slot_map=page * P + pos % P, k_new=k_new, v_new=v_new, rows=T,
                  workspace=torch.zeros(256, dtype=torch.uint8, **dev))
        return st
    hq = case["hq"]
    st.update(q=values(T, hq, d).to(dt), out=torch.empty(T, hq, d, dtype=dt, **dev),
              lse=torch.empty(T, hq, dtype=torch.float32, **dev), max_q=max(new), max_pages=max(pages))
    if own:
        # the step's plan: made once for the step's lengths and kept for all of the model's layers
        from paged_kv_attention_27_gb300 import binding as B
        import numpy as np
        prefill = case["op"] == "prefill"
        st["plan"] = B.fi_plan(
            B.FI_MODE_PREFILL if prefill else B.FI_MODE_DECODE, case["batch"],
            np.array(qo) if prefill else None, np.array(indptr), last.cpu().numpy(), hq, hkv, d, P,
            prefill, {"window_left": case["window"], "kv_dtype": B.FI_DTYPE_E4M3_PAGE,
                      "dtype": B.FI_DTYPE_BF16 if case["dtype"] == "bf16" else B.FI_DTYPE_FP16},
            torch.cuda.get_device_properties(0).multi_processor_count)
        st["workspace"] = torch.empty(max(st["plan"].workspace_bytes, 256), dtype=torch.uint8, **dev)
    return st


# ---- the operators ------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if case["op"] == "table":
        (_own_table if own else _plain_table)(state)
        return {k: state[k] for k in ("kv_len_out", "ring_state_out", "table", "ring", "page_indptr",
                                      "page_indices", "last_page_len", "qo_indptr", "slot_map",
                                      "positions")}
    if case["op"] == "append":
        if own:
            _own_append(state)
        else:
            _plain_append(state["k_new"], state["k"], state["k_scale"], state["slot_map"], case)
            _plain_append(state["v_new"], state["v"], state["v_scale"], state["slot_map"], case)
        f8 = torch.float8_e4m3fn
        return {"k": state["k"].view(f8), "v": state["v"].view(f8), "k_scale": state["k_scale"],
                "v_scale": state["v_scale"]}
    out, lse = _own_attention(state) if own else _plain_attention(state)
    return {"out": out, "lse": lse}


def _own_table(s):
    from paged_kv_attention_27_gb300 import binding as B
    c = s["case"]
    B.fi_page_table_step(c["batch"], s["slots"], s["new_len"], c["max_requests"],
                         s["table"].shape[1], c["page"], s["kv_len"], s["kv_len_out"], s["table"],
                         s["ring"], s["ring"].numel(), s["ring_state"], s["ring_state_out"],
                         s["page_indptr"], s["page_indices"], s["page_indices"].numel(),
                         s["last_page_len"], s["qo_indptr"], s["slot_map"], s["positions"],
                         s["slot_map"].numel(), s["workspace"], 256)


def _own_append(s):
    from paged_kv_attention_27_gb300 import binding as B
    c = s["case"]
    B.fi_append_paged_kv(s["rows"], s["slot_map"], s["k_new"], s["v_new"], s["k_new"].stride(0),
                         B.FI_DTYPE_BF16 if c["dtype"] == "bf16" else B.FI_DTYPE_FP16, c["hkv"],
                         c["d"], s["k"], s["v"], B.FI_DTYPE_E4M3_PAGE, B.LAYOUTS[c["layout"]], 0,
                         s["num_pages"], c["page"], s["k_scale"], s["v_scale"], s["workspace"], 256)


def _own_attention(s):
    from paged_kv_attention_27_gb300 import binding as B
    c = s["case"]
    tables = (s["page_indptr"], s["page_indices"], s["last_page_len"])
    rest = (1.0 / math.sqrt(c["d"]), 1.0, 1.0, s["out"], s["lse"], s["workspace"])
    scales = dict(k_head_scale=s["k_scale"], v_head_scale=s["v_scale"])
    layout = B.LAYOUTS[c["layout"]]
    if c["op"] == "decode":
        B.fi_batch_decode_paged(s["plan"], s["q"], s["k"], s["v"], layout, 0, s["num_pages"],
                                *tables, *rest, **scales)
    else:
        B.fi_batch_prefill_paged(s["plan"], s["q"], s["qo_indptr"], s["k"], s["v"], layout, 0,
                                 s["num_pages"], *tables, *rest, **scales)
    return s["out"], s["lse"]


def _owner(ends, n):
    """For each of n consecutive items: the row whose range [ends[r-1], ends[r]) holds it (the last
    row's number + 1 behind the last range), and the item's number."""
    i = torch.arange(n, device=ends.device)
    return torch.searchsorted(ends, i, right=True), i


def _plain_table(s):
    """With a request's length L before the step and L' = L + new (new < 0 drops tokens, a negative
    slot is a padding row): its pages are the first ceil(L' / P) of its row of the table. The pages
    it lacks come from the head of the ring in batch order, those it no longer needs go to its tail."""
    c, P = s["case"], s["case"]["page"]
    table, ring = s["table"], s["ring"]
    cap = ring.numel()
    real = s["slots"] >= 0
    slot = s["slots"].clamp(min=0).long()
    old = torch.where(real, s["kv_len"][slot], 0).long()
    new = torch.where(real, s["new_len"], 0).long()
    cur = old + new
    had, has = (old + P - 1) // P, (cur + P - 1) // P
    take, give, rows = (has - had).clamp(min=0), (had - has).clamp(min=0), new.clamp(min=0)
    head, count = s["ring_state"].long().unbind()
    ends = {k: torch.cumsum(v, 0) for k, v in (("take", take), ("give", give), ("has", has), ("rows", rows))}
    last = c["batch"] - 1
    n_rows = s["slot_map"].numel()
    # pages taken: at most as many as the step's rows
    r, i = _owner(ends["take"], n_rows)
    ok, r = i < ends["take"][-1], r.clamp(max=last)
    at = had[r] + i - (ends["take"] - take)[r]
    table[slot[r[ok]], at[ok]] = ring[(head + i[ok]) % cap]
    # pages returned
    r, i = _owner(ends["give"], cap)
    ok, r = i < ends["give"][-1], r.clamp(max=last)
    at = has[r] + i - (ends["give"] - give)[r]
    ring[(head + count + i[ok]) % cap] = table[slot[r[ok]], at[ok]]
    # the step's page table
    r, i = _owner(ends["has"], s["page_indices"].numel())
    ok, r = i < ends["has"][-1], r.clamp(max=last)
    at = (i - (ends["has"] - has)[r])[ok]
    s["page_indices"][ok] = table[slot[r[ok]], at]
    s["page_indptr"][0] = 0
    s["page_indptr"][1:] = ends["has"].to(INT)
    s["last_page_len"].copy_(torch.where(cur > 0, (cur - 1) % P + 1, 0))
    s["qo_indptr"][0] = 0
    s["qo_indptr"][1:] = ends["rows"].to(INT)
    # where each new row goes
    r, i = _owner(ends["rows"], n_rows)
    ok, r = i < ends["rows"][-1], r.clamp(max=last)
    pos = torch.where(ok, old[r] + i - (ends["rows"] - rows)[r], 0)
    page = table[slot[r], pos // P].long()
    s["slot_map"].copy_(torch.where(ok, page * P + pos % P, -1))
    s["positions"].copy_(pos)
    s["kv_len_out"][slot[real]] = cur[real].to(INT)
    s["ring_state_out"][0] = ((head + ends["take"][-1]) % cap).to(INT)
    s["ring_state_out"][1] = (count - ends["take"][-1] + ends["give"][-1]).to(INT)


def _plain_append(rows, cache, scale, slot_map, case):
    """For every (page, head) with new rows: s' = the smallest power of two with amax <= 448 s' over
    them (finite values only); the page's scale becomes max(old, s'), or s' where the first new row
    is the page's first. Codes of older rows are rounded again where the scale grew; the new rows'
    are x / scale, rounded to nearest even (NaN and infinities give NaN)."""
    P, hkv, d = case["page"], case["hkv"], case["d"]
    n = scale.shape[0]
    x = rows.reshape(rows.shape[0], hkv, d).float()
    page, at = slot_map // P, slot_map % P
    amax = torch.where(x.isfinite(), x.abs(), 0).amax(dim=2)
    most = torch.zeros(n, hkv, device=x.device).scatter_reduce_(
        0, page[:, None].expand(-1, hkv), amax, "amax")
    first = torch.full((n,), P, device=x.device).scatter_reduce_(0, page, at, "amin")
    hit = (first < P).nonzero()[:, 0]
    fresh = (first[hit] == 0)[:, None]
    grown = _scale_of(most[hit])
    before = scale[hit]
    after = torch.where(fresh, grown, torch.maximum(before, grown))
    scale[hit] = after
    view = cache if case["layout"] == "NHD" else cache.transpose(1, 2)   # [page][slot][head][dim]
    codes = view[hit]
    again = (codes.view(torch.float8_e4m3fn).float() * (before / after)[:, None, :, None])
    again = again.to(torch.float8_e4m3fn).view(torch.uint8)
    older = torch.arange(P, device=x.device)[None, :] < first[hit][:, None]
    change = older[:, :, None] & (after > before)[:, None, :] & ~fresh[:, None, :]
    view[hit] = torch.where(change[..., None], again, codes)
    view[page, at] = (x / scale[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _bounds(case, ctx, rows_at, total):
    """Keys a row sees: [lo, hi) for the row at key position ctx + rows_at."""
    pos = ctx + rows_at
    lo = (pos - case["window"]).clamp(min=0) if case["window"] >= 0 else torch.zeros_like(pos)
    return lo, torch.minimum(pos + 1, total)


def _plain_attention(s):
    """softmax(scale q k^T) v with k and v the codes times their page's scale, all requests padded
    to the longest."""
    c = s["case"]
    n, hq, hkv, d, P = c["batch"], c["hq"], c["hkv"], c["d"], c["page"]
    g, mq, mp = hq // hkv, s["max_q"], s["max_pages"]
    dev = s["q"].device
    has = (s["page_indptr"][1:] - s["page_indptr"][:-1]).long()
    total = (has - 1) * P + s["last_page_len"]
    rows = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    j = torch.arange(mp, device=dev)[None]
    at = s["page_indptr"][:-1].long()[:, None] + torch.minimum(j, has[:, None] - 1)
    pages = s["page_indices"][at].long()                               # [n][mp]

    def cache(codes, scale):
        x = codes[pages].view(torch.float8_e4m3fn).float()              # [n][mp] + a page
        x = x if c["layout"] == "HND" else x.transpose(2, 3)            # [n][mp][hkv][P][d]
        x = x * scale[pages][..., None, None]
        return x.transpose(1, 2).reshape(n, hkv, mp * P, d)

    i = torch.arange(mq, device=dev)[None]
    take = s["qo_indptr"][:-1].long()[:, None] + torch.minimum(i, rows[:, None] - 1)
    q = s["q"][take].float().reshape(n, mq, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, mq * g, d)
    x = torch.matmul(q, cache(s["k"], s["k_scale"]).transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    lo, hi = _bounds(c, (total - rows)[:, None], torch.minimum(i, rows[:, None] - 1), total[:, None])
    t = torch.arange(mp * P, device=dev)
    hide = (t < lo[..., None]) | (t >= hi[..., None])                  # [n][mq][keys]
    x = x.view(n, hkv, mq, g, mp * P).masked_fill_(hide[:, None, :, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    x = x.sub_(top).exp_()
    total_w = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x.view(n, hkv, mq * g, mp * P), cache(s["v"], s["v_scale"]))
    o = (o.view(n, hkv, mq, g, d) / total_w).permute(0, 2, 1, 3, 4).reshape(n, mq, hq, d)
    lse = (top + total_w.log())[..., 0].permute(0, 2, 1, 3).reshape(n, mq, hq)
    real = i < rows[:, None]
    s["out"].copy_(o[real])
    s["lse"].copy_(lse[real])
    return s["out"], s["lse"]


# ---- what a pass cannot do without --------------------------------------------------------------
def work(case):
    ctx, new = _lens(case)
    P = case["page"]
    if case["op"] == "table":
        rng = random.Random(case["lens"] + 1)
        live = [rng.random() >= case["pad"] for _ in range(case["batch"])]
        live[0] = True
        after = sum(-(-(c + x) // P) for c, x, ok in zip(ctx, new, live) if ok)
        rows = sum(max(x, 0) for x, ok in zip(new, live) if ok) + 16
        # lengths and slots in, offsets and lengths out, table entries in and out, rows' slots
        return {"bytes": 28 * case["batch"] + 8 * after + 12 * rows, "flops": 0}
    elem = case["hkv"] * case["d"]
    if case["op"] == "append":
        rows = sum(new)
        touched = sum(-(-(c + x) // P) - c // P for c, x in zip(ctx, new))
        return {"bytes": rows * (elem * 6 + 8) + touched * case["hkv"] * 16, "flops": rows * elem * 4}
    keys = pairs = pages = 0
    for c, x in zip(ctx, new):
        w = case["window"]
        first = max(0, c - w) if w >= 0 else 0
        keys += c + x - first
        pages += -(-(c + x) // P) - first // P
        pairs += sum(min(c + r + 1, w + 1 if w >= 0 else c + r + 1) for r in range(x))
    q = sum(new) * case["hq"]
    return {"bytes": keys * elem * 2 + pages * case["hkv"] * 8 + q * case["d"] * 4 + q * 4,
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ---- the definition in 64 bits ------------------------------------------------------------------
def _grid():
    """The non-negative finite E4M3 values in order of their codes."""
    return torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def _nearest(x, grid):
    """x (finite) to the nearest value of the grid, ties to the even code."""
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a).clamp(1, 126)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], x)


def _exact_append(rows, codes, scale, slot_map, case):
    P, hkv, d = case["page"], case["hkv"], case["d"]
    grid = _grid().to(rows.device)
    value = codes.view(torch.float8_e4m3fn).double()
    value = value.clone() if case["layout"] == "NHD" else value.transpose(1, 2).clone()
    scale = scale.double().clone()
    slots = slot_map.tolist()
    x = rows.double().reshape(-1, hkv, d)
    # runs of rows of one page
    starts = [t for t in range(len(slots)) if t == 0 or slots[t] // P != slots[t - 1] // P]
    for t0, t1 in zip(starts, starts[1:] + [len(slots)]):
        page, first = slots[t0] // P, slots[t0] % P
        y = x[t0:t1]
        amax = y.abs().amax(dim=(0, 2))
        s = torch.exp2(torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** MIN_EXP))))
        s = torch.where(amax / 448 <= s / 2, s / 2, s).clamp(min=2.0 ** MIN_EXP)
        if first:
            s = torch.maximum(s, scale[page])
            value[page, :first] = _nearest(value[page, :first] * (scale[page] / s)[None, :, None], grid)
        scale[page] = s
        value[page, first:first + t1 - t0] = _nearest(y / s[None, :, None], grid)
    return value if case["layout"] == "NHD" else value.transpose(1, 2).contiguous(), scale


def exact(case, seed):
    if case["op"] == "table":
        return None
    if case["op"] == "append":
        ctx, new = _lens(case)
        if sum(-(-x // case["page"]) + 1 for x in new) > 6000:
            return None
        s = prepare(case, seed)
        k, ks = _exact_append(s["k_new"], s["k"], s["k_scale"], s["slot_map"], case)
        v, vs = _exact_append(s["v_new"], s["v"], s["v_scale"], s["slot_map"], case)
        return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}
    if work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    ctx, new = _lens(case)
    g = hq // hkv
    out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), hq), -math.inf, dtype=torch.float64, device="cuda")
    starts, r0 = s["page_indptr"].tolist(), 0
    for b in range(case["batch"]):
        ids = s["page_indices"][starts[b]:starts[b + 1]].long()
        n, m = ctx[b] + new[b], new[b]
        kv = []
        for codes, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            x = codes[ids].view(torch.float8_e4m3fn).double()
            x = x if case["layout"] == "NHD" else x.transpose(1, 2)
            kv.append((x * scale[ids].double()[:, None, :, None]).reshape(-1, hkv, d)[:n])
        pos = torch.arange(ctx[b], n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        seen = t <= pos
        if case["window"] >= 0:
            seen &= t >= pos - case["window"]
        for h in range(hkv):
            q = s["q"][r0:r0 + m, h * g:(h + 1) * g].double()
            x = torch.einsum("mgd,nd->gmn", q, kv[0][:, h]) * (1.0 / math.sqrt(d))
            x = torch.where(seen, x, -math.inf)
            l = torch.logsumexp(x, dim=2)
            p = torch.exp(x - l[..., None])
            out[r0:r0 + m, h * g:(h + 1) * g] = torch.einsum("gmn,nd->mgd", p, kv[1][:, h])
            lse[r0:r0 + m, h * g:(h + 1) * g] = l.T
        r0 += m
    return {"out": out, "lse": lse}
