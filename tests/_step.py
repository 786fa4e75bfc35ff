"""Plain implementations of a serving step's preparation, for the tests: the
page-table step in Python integers, the quantising append in float64."""
import numpy as np

MIN_EXP = -100


class StepError(Exception):
    pass


def page_table_step(slots, new_len, kv_len, table, ring, ring_state, page_size, page_capacity,
                    token_capacity):
    """The step on copies of its arrays; returns a dict of every output, or
    raises StepError where the step cannot be made."""
    P, cap, max_pages = page_size, len(ring), table.shape[1]
    kv_len, table, ring = kv_len.copy(), table.copy(), ring.copy()
    head, count = int(ring_state[0]), int(ring_state[1])
    named = [s for s in slots if s >= 0]
    if len(set(named)) < len(named) or any(s >= len(kv_len) for s in named):
        raise StepError("bounds")
    taken, given, indptr, indices, last, qo, smap, pos = [], [], [0], [], [], [0], [], []
    after = {}
    for s, n in zip(slots, new_len):
        if s < 0:
            indptr.append(indptr[-1])
            last.append(0)
            qo.append(qo[-1])
            continue
        old, n = int(kv_len[s]), int(n)
        length = old + n
        if length < 0:
            raise StepError("bounds")
        if length > max_pages * P:
            raise StepError("pages")
        had, has = -(-old // P), -(-length // P)
        row = table[s].copy()
        for j in range(had, has):
            i = len(taken)
            if i >= count:
                raise StepError("pages")
            row[j] = ring[(head + i) % cap]
            taken.append(row[j])
        given += [row[j] for j in range(has, had)]
        after[s] = (length, row)
        indices += row[:has].tolist()
        indptr.append(indptr[-1] + has)
        last.append((length - 1) % P + 1 if length else 0)
        qo.append(qo[-1] + max(n, 0))
        for i in range(max(n, 0)):
            p = old + i
            pos.append(p)
            smap.append(int(row[p // P]) * P + p % P)
    if len(indices) > page_capacity or len(smap) > token_capacity:
        raise StepError("pages")
    if count + len(given) > cap:
        raise StepError("bounds")
    for i, page in enumerate(given):
        ring[(head + count + i) % cap] = page
    for s, (length, row) in after.items():
        kv_len[s] = length
        table[s] = row
    return dict(kv_len=kv_len, block_table=table, free_ring=ring,
                ring_state=np.array([(head + len(taken)) % cap, count - len(taken) + len(given)]),
                page_indptr=np.array(indptr), page_indices=np.array(indices, dtype=np.int64),
                last_page_len=np.array(last), qo_indptr=np.array(qo),
                slot_map=np.array(smap + [-1] * (token_capacity - len(smap))),
                positions=np.array(pos + [0] * (token_capacity - len(pos))))


_GRID = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                  for e in range(16) for m in range(8)][:127])


def e4m3_value(codes):
    """E4M3 codes -> float64 values (NaN for 0x7f and 0xff)."""
    c = np.asarray(codes, dtype=np.uint8)
    v = np.append(_GRID, np.nan)[c & 0x7f]
    return np.where(c & 0x80, -v, v)


def e4m3_code(x):
    """float64 -> E4M3 codes, to nearest, ties to the even code; saturated;
    NaN and infinities give 0x7f (the sign of a NaN is not defined)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0)), 448.0)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 126)
    lo = hi - 1
    up, down = _GRID[hi] - a, a - _GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code = np.where(np.isfinite(x), code | (np.signbit(x) * np.uint8(0x80)), np.uint8(0x7f))
    return code.astype(np.uint8)


def scale_of(amax):
    """The smallest power of two s >= 2^MIN_EXP with amax <= 448 s."""
    k = MIN_EXP
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append_page_scaled(slot_map, x, cache, scale, page_size):
    """x [rows][heads][dim] float64 into copies of cache [page][slot][head][dim]
    (codes) and scale [page][head]; returns both."""
    cache, scale = cache.copy(), scale.astype(np.float64)
    P, t, n = page_size, 0, len(slot_map)
    while t < n:
        s = int(slot_map[t])
        if s < 0 or s >= cache.shape[0] * P:
            t += 1
            continue
        m = 1
        while t + m < n and (s + m) % P and slot_map[t + m] == s + m:
            m += 1
        page, first = s // P, s % P
        for h in range(cache.shape[2]):
            y = x[t:t + m, h]
            fine = np.abs(y[np.isfinite(y)])
            new = scale_of(fine.max() if fine.size else 0.0)
            old = scale[page, h]
            if first and old >= new:
                new = old
            elif first:
                older = e4m3_value(cache[page, :first, h])
                cache[page, :first, h] = e4m3_code(older * (old / new))
            scale[page, h] = new
            cache[page, first:first + m, h] = e4m3_code(y / new)
        t += m
    return cache, scale
