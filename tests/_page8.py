"""Batches over a page-scaled FP8 cache for the tests: seeded inputs, a plain
float64 implementation of the attention with the quantities its error bound is
made of, and the comparison.

The bound on out, per element (h = half a step of the output type relative to
the value, eps / 2; a = sum p |v| over the row's keys, p normalised):
    h |o|                       rounding the output
  + r a                         the weights as sums of e4m3 terms: two terms of
                                4 bits each round a weight by at most 2^-8 of
                                itself, three (fp16) by 2^-12; 16-bit weights
                                (prefill) by at most 2^-8 (bf16) and 2^-11
  + n u vmax pmax               weights so small that their last term is
                                subnormal: at most u of the largest weight.
                                Decode stores a weight w <= 2^4 as terms of
                                16 w, the second times 16, the third times 256:
                                half of E4M3's step of 2^-9 is 2^-10 / 256 =
                                2^-18 of a weight of 1 (two terms) or 2^-22
                                (three); the running maximum is within a factor
                                of 2^4 of the largest weight, which is >= 1 when
                                it is set. Prefill's fp16 weights: 2^-25.
  + 2 d (a + |o|)               d: the error of the scores (below), which is a
                                relative error of each weight and of their sum
The fp32 sums of a score's head_dim products (times the fp32 roundings of the
scales) are off by at most (head_dim + 8) 2^-24 of sum |q k|; the exponentials
of ex2.approx by 2^-22: d = (head_dim + 8) 2^-24 max sum |q k| sm_scale +
2^-20. To d also belong q's elements that E4M3's finest step rounds: q enters
as terms of x = q times a power of two with the row's largest |x| in 224..448;
prefill's terms are exact down to the step 2^-9, so an element of bf16 (8 bits)
is exact from |x| = 2^-2 on, of fp16 (11 bits, three terms) from 2 on, and one
below is off by at most 2^-10; decode's last term is scaled by 16 (256), so
its elements are exact from 2^-6 (2^-7) on and off by at most 2^-14 (2^-18):
+ sm_scale max_t sum_e off_e |k_te|. The bound on lse is d + 2^-22 |lse|."""
import numpy as np

from . import _step


class Batch:
    """q bits, codes and scales on the host. qo_lens: rows per request (None:
    one each, a decode batch)."""

    def __init__(self, kv_lens, hq, hkv, d, P, layout="NHD", dtype="bf16", qo_lens=None,
                 causal=True, window=-1, seed=0, scales="pow2", spare=3, tail=None, v_spread=0):
        rng = np.random.default_rng(seed)
        self.kv_lens, self.hq, self.hkv, self.d, self.P = list(kv_lens), hq, hkv, d, P
        self.layout, self.dtype, self.window = layout, dtype, window
        self.decode = qo_lens is None
        self.qo_lens = [1] * len(kv_lens) if self.decode else list(qo_lens)
        self.causal = causal and not self.decode
        pages = [-(-n // P) for n in kv_lens]
        self.page_indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.num_pages = int(self.page_indptr[-1]) + spare
        self.page_indices = rng.permutation(self.num_pages)[:self.page_indptr[-1]].astype(np.int32)
        self.last_page_len = np.array([(n - 1) % P + 1 if n else 0 for n in kv_lens], dtype=np.int32)
        self.qo_indptr = np.concatenate([[0], np.cumsum(self.qo_lens)]).astype(np.int32)
        self.rows = int(self.qo_indptr[-1])
        self.sm_scale = 1.0 / np.sqrt(d)
        self.q = _as16(rng.standard_normal((self.rows, hq, d)), dtype)
        shape = (self.num_pages, P, hkv, d)
        self.codes, self.scale = [], []
        for which in range(2):
            x = rng.standard_normal(shape)
            if which == 1 and v_spread:      # pages of very unequal values
                x = x * np.exp2(rng.integers(-v_spread, v_spread + 1, (self.num_pages, 1, hkv, 1)))
            amax = np.abs(x).max(axis=(1, 3))
            if scales == "pow2":
                s = np.exp2(np.ceil(np.log2(amax / 448)))
            else:                            # any scale, as of another quantiser
                s = (amax / 448 * rng.uniform(1, 3, amax.shape)).astype(np.float32).astype(np.float64)
            self.codes.append(_step.e4m3_code(x / s[:, None, :, None]))
            self.scale.append(s)
        if tail is not None:                 # slots no request uses
            used = np.zeros((self.num_pages, P), dtype=bool)
            for b, n in enumerate(kv_lens):
                for t in range(n):
                    used[self.page_indices[self.page_indptr[b] + t // P], t % P] = True
            for c in self.codes:
                c[~used] = tail

    def q64(self):
        return _from16(self.q, self.dtype)

    def kv64(self, which):
        v = _step.e4m3_value(self.codes[which])
        return v * self.scale[which][:, None, :, None]

    def plan(self, B, sms=None, num_sms=None):
        prefill = not self.decode
        return B.fi_plan(B.FI_MODE_PREFILL if prefill else B.FI_MODE_DECODE, len(self.kv_lens),
                         self.qo_indptr if prefill else None, self.page_indptr, self.last_page_len,
                         self.hq, self.hkv, self.d, self.P, self.causal,
                         {"window_left": self.window, "kv_dtype": B.FI_DTYPE_E4M3_PAGE,
                          "dtype": B.FI_DTYPE_BF16 if self.dtype == "bf16" else B.FI_DTYPE_FP16},
                         sms or num_sms or 152)


def _as16(x, dtype):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float16)


def _from16(t, dtype):
    return t.double().numpy()


class Device:
    """A batch on the GPU, its plan, outputs and workspace."""

    def __init__(self, b, sms=None, device="cuda"):
        import torch

        from paged_kv_attention_27_gb300 import binding as B
        self.b, self.B = b, B
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
        lay = (lambda a: a) if b.layout == "NHD" else (lambda a: a.transpose(0, 2, 1, 3))
        self.q = b.q.to(device)
        self.k, self.v = [dev(lay(c)) for c in b.codes]
        self.ks, self.vs = [dev(s.astype(np.float32)) for s in b.scale]
        self.page_indptr, self.last_page_len = dev(b.page_indptr), dev(b.last_page_len)
        self.page_indices = dev(b.page_indices if len(b.page_indices) else np.zeros(1, np.int32))
        self.qo_indptr = dev(b.qo_indptr)
        self.plan = b.plan(B, sms, torch.cuda.get_device_properties(device).multi_processor_count)
        self.workspace = torch.empty(max(self.plan.workspace_bytes, 256), dtype=torch.uint8, device=device)
        self.out = torch.full((b.rows, b.hq, b.d), float("nan"), dtype=b.q.dtype, device=device)
        self.lse = torch.full((b.rows, b.hq), float("nan"), dtype=torch.float32, device=device)

    def run(self, k_scale=1.0, v_scale=1.0, stream=None, page_stride=0, lse=True):
        b, B = self.b, self.B
        tables = (self.page_indptr, self.page_indices, self.last_page_len, b.sm_scale, k_scale,
                  v_scale, self.out, self.lse if lse else None, self.workspace)
        cache = (self.k, self.v, B.LAYOUTS[b.layout], page_stride, b.num_pages)
        kw = dict(stream=stream, k_head_scale=self.ks, v_head_scale=self.vs)
        if b.decode:
            B.fi_batch_decode_paged(self.plan, self.q, *cache, *tables, **kw)
        else:
            B.fi_batch_prefill_paged(self.plan, self.q, self.qo_indptr, *cache, *tables, **kw)
        return self.out, self.lse

    def status(self):
        return self.B.fi_check_device_status(self.workspace)


def reference(b, requests=None, k_scale=1.0, v_scale=1.0):
    """out, lse and the parts of the bound (a, vmax * pmax * n, d), float64."""
    q, k, v = b.q64(), b.kv64(0) * k_scale, b.kv64(1) * v_scale
    out, a = np.zeros((b.rows, b.hq, b.d)), np.zeros((b.rows, b.hq, b.d))
    lse = np.full((b.rows, b.hq), -np.inf)
    tiny, ds = np.zeros((b.rows, b.hq)), np.zeros((b.rows, b.hq))
    g = b.hq // b.hkv
    for r, n in enumerate(b.kv_lens):
        if requests is not None and r not in requests:
            continue
        m, r0 = b.qo_lens[r], int(b.qo_indptr[r])
        if n == 0 or m == 0:
            continue
        t = np.arange(n)
        pages = b.page_indices[b.page_indptr[r] + t // b.P]
        pos = n - m + np.arange(m)[:, None]
        vis = (t <= pos) if b.causal else np.ones((m, n), dtype=bool)
        if b.window >= 0:
            vis = vis & (t >= pos - b.window)
        for h in range(b.hq):
            kk, vv = k[pages, t % b.P, h // g], v[pages, t % b.P, h // g]
            qq = q[r0:r0 + m, h]
            s = np.where(vis, b.sm_scale * (qq @ kk.T), -np.inf)
            top = s.max(axis=1, keepdims=True)
            some = np.isfinite(top[:, 0])
            with np.errstate(invalid="ignore"):
                p = np.where(vis, np.exp(s - np.where(some[:, None], top, 0)), 0)
                l = p.sum(axis=1, keepdims=True)
                p = np.where(some[:, None], p / np.where(l == 0, 1, l), 0)
                lse[r0:r0 + m, h] = np.where(some, top[:, 0] + np.log(np.where(l[:, 0] == 0, 1, l[:, 0])), -np.inf)
            out[r0:r0 + m, h] = p @ vv
            a[r0:r0 + m, h] = p @ np.abs(vv)
            # weights enter times their page's value scale: p |v| at its largest
            tiny[r0:r0 + m, h] = n * (p * np.abs(vv).max(axis=1)[None]).max(axis=1)
            fine, off = {(True, "bf16"): (-6, -14), (True, "fp16"): (-7, -18),
                         (False, "bf16"): (-2, -10), (False, "fp16"): (1, -10)}[b.decode, b.dtype]
            unit = np.abs(qq).max(axis=1, keepdims=True) / 224       # at least x's unit
            off_q = np.where(np.abs(qq) < unit * 2.0 ** fine, unit * 2.0 ** off, 0)
            ds[r0:r0 + m, h] = (b.sm_scale * np.where(vis, off_q @ np.abs(kk).T, 0).max(axis=1) +
                                (b.d + 8) * 2.0 ** -24 * b.sm_scale *
                                np.where(vis, np.abs(qq) @ np.abs(kk).T, 0).max(axis=1) + 2.0 ** -20)
    return out, lse, a, tiny, ds


def compare(b, out, lse, ref, rows=None, what=""):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ro, rl, a, tiny, ds = ref
    if rows is not None:
        o, l, ro, rl, a, tiny, ds = [x[rows] for x in (o, l, ro, rl, a, tiny, ds)]
    h, r, u = (2.0 ** -8, 2.0 ** -8, 2.0 ** -18) if b.dtype == "bf16" else (2.0 ** -11, 2.0 ** -11, 2.0 ** -22)
    bound = h * np.abs(ro) + r * a + u * tiny[..., None] + 2 * ds[..., None] * (a + np.abs(ro))
    assert np.all(np.isfinite(o)), f"{what}: non-finite output"
    err = np.abs(o - ro)
    over = err > bound
    print(f"{what}: out max {err.max():.2e}, {np.max(err / np.maximum(bound, 1e-300)):.2f} of its bound")
    assert not over.any(), (f"{what}: {over.sum()} of {over.size} outputs over the bound, worst at "
                            f"{np.unravel_index(np.argmax(err - bound), err.shape)}")
    assert np.array_equal(np.isneginf(l), np.isneginf(rl)), f"{what}: -inf lse pattern"
    fin = np.isfinite(rl)
    le = np.abs(l[fin] - rl[fin])
    lb = ds[fin] + 2.0 ** -22 * np.abs(rl[fin])
    if le.size:
        print(f"{what}: lse max {le.max():.2e}, {np.max(le / lb):.2f} of its bound")
        assert np.all(le <= lb), f"{what}: lse over its bound"
