"""Helpers of the paged cache's tests: batches over shuffled pages, and the operators' definitions in
64 bits on the CPU, one row at a time.

Tolerances, from the formats (half a step of bf16 is 2^-8 relative, of fp32 2^-24):
  * read back: one rounding to bf16 of an fp32 product, 2^-8 + 2^-24 relative;
  * a score s = scale * q . k: fp32 sums of D exact products in any order, D * 2^-24 of the sum of their
    magnitudes, and 4 * 2^-24 of |s| for the scalings; over an e4m3 cache the queries are represented
    to 2^-17 of the row's largest magnitude;
  * attention: with every score off by at most ds, each weight exp(s - m) is off by the factor
    exp(+-2 ds) (m moves with them), by 2^-20 for the exponential itself, and by one rounding to bf16
    (2^-8) where it meets V; the sums of n terms add n * 2^-24; the result is rounded to bf16 once. All
    but the last count relative to sum p |v|;
  * lse: ds + 2^-20 + n * 2^-24 and 4 * 2^-24 of its own magnitude.
"""
import math

import torch

from mixture_experts_ffn_router_gb300 import binding as B

BF = 2.0 ** -8
F32 = 2.0 ** -24


class Case:
    """Sequences with `new` new tokens each, the last of their `kv` cached ones, in shuffled pages."""

    def __init__(self, fmt, hq, hkv, d, page, new, kv, seed=0, pad_rows=0, garbage="nan", device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.hq, self.hkv, self.d, self.page = fmt, hq, hkv, d, page
        self.new, self.kv, self.device = list(new), list(kv), device
        n_of = [-(-max(n, 0) // page) for n in kv]
        self.n_pages = sum(n_of) + 3
        order = torch.randperm(self.n_pages, generator=g).tolist()
        cols = max(n_of + [1])
        # Entries past a sequence's last page are not ids of anything.
        self.pages = torch.full((len(kv), cols), -7, dtype=torch.int32)
        for b, n in enumerate(n_of):
            for i in range(n):
                self.pages[b, i] = order.pop()
        self.cu = [0]
        for n in new:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1] + pad_rows
        # Every sequence's whole history, as bf16.
        self.k, self.v = ([torch.randn(max(n, 0), hkv, d, generator=g).to(torch.bfloat16) for n in kv]
                          for _ in range(2))
        self.q = (torch.randn(self.T, hq, d, generator=g) * 1.5).to(torch.bfloat16)
        self.garbage = garbage

    def handle(self, **kw):
        return B.PagedKV(self.hq, self.hkv, self.d, self.page, self.n_pages, self.fmt, max_tokens=max(self.T, 1, sum(
            max(n, 0) for n in self.kv)), max_seqs=max(len(self.kv), 1), **kw)

    def batch(self, new=None):
        new = self.new if new is None else new
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        return B.KVBatch(cu.to(self.device), torch.tensor(self.kv, dtype=torch.int32).to(self.device),
                         self.pages.to(self.device), max_new=max(new + [0]))

    def empty_cache(self, kv):
        """A cache full of garbage, as memory is before it is written."""
        c = kv.new_cache()
        if self.garbage == "nan":
            if self.fmt == "bf16":
                c.k.fill_(math.nan)
                c.v.fill_(math.nan)
            else:
                for t in (c.k, c.v):
                    t.view(torch.uint8).fill_(0x7f)
                c.k_scale.fill_(math.nan)
                c.v_scale.fill_(math.inf)
        return c

    def filled(self, kv):
        """A cache that holds every sequence's history, written in one call."""
        c = self.empty_cache(kv)
        whole = [max(n, 0) for n in self.kv]
        if sum(whole):
            kv.write(c, self.batch(whole), torch.cat(self.k).to(self.device), torch.cat(self.v).to(self.device))
        return c

    def stored(self, name, b):
        """What the cache holds of sequence b, in 64 bits."""
        x = (self.k if name == "k" else self.v)[b]
        return dequantised(x)[0] if self.fmt == "e4m3" else x.double()


def quantised(x):
    """Codes (as values) and fp32 scales of bf16 rows, by the format's rule."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = torch.where(torch.isfinite(amax), amax / 448.0, torch.full_like(amax, math.nan))
    codes = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return codes.to(torch.float8_e4m3fn), scale


def dequantised(x):
    codes, scale = quantised(x)
    return codes.double() * scale.double()[..., None], scale


def visible(p, window, sinks):
    """Positions a token at position p sees."""
    return [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]


def attention(case, scale=None, window=0, sinks=0):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
    scale = case.d ** -0.5 if scale is None else scale
    out = torch.zeros(case.T, case.hq, case.d, dtype=torch.float64)
    lse = torch.full((case.T, case.hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    g = case.hq // case.hkv
    for b, n in enumerate(case.new):
        k, v = case.stored("k", b), case.stored("v", b)
        for i in range(n):
            row, p = case.cu[b] + i, case.kv[b] - n + i
            at = torch.tensor(visible(p, window, sinks), dtype=torch.long)
            if not len(at):
                continue
            for h in range(case.hkv):
                q = case.q[row, h * g:(h + 1) * g].double()
                kk, vv = k[at, h], v[at, h]
                s = scale * q @ kk.T
                ds = case.d * F32 * scale * (q.abs() @ kk.abs().T) + 4 * F32 * s.abs()
                if case.fmt == "e4m3":
                    ds = ds + 2.0 ** -17 * scale * q.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)
                ds = ds.amax(-1, keepdim=True)
                w = torch.softmax(s, -1)
                hs = slice(h * g, (h + 1) * g)
                out[row, hs] = w @ vv
                lse[row, hs] = torch.logsumexp(s, -1)
                rel = torch.expm1(2 * ds) + 2.0 ** -20 + BF + 2 * len(at) * F32
                tol[row, hs] = rel * (w @ vv.abs()) * (1 + BF) + BF * out[row, hs].abs()
                ltol[row, hs] = ds[:, 0] + 2.0 ** -20 + len(at) * F32 + 4 * F32 * lse[row, hs].abs()
    return out, lse, tol, ltol


def check_close(got, want, tol, label=""):
    got = got.double().cpu()
    assert got.shape == want.shape
    for name, f in (("NaN", torch.isnan), ("infinity", torch.isinf)):
        bad = (f(got) != f(want)).nonzero()
        assert not len(bad), "%s %s at %s, or missing there" % (label, name, bad[0].tolist())
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), label
    fine = torch.isfinite(want)
    over = ((got - want).abs() - tol)[fine]
    assert not len(over) or over.max() <= 0, "%s off by %.3e more than allowed (%d of %d values)" % (
        label, over.max(), (over > 0).sum(), over.numel())


def check_attention(case, window=0, sinks=0, scale=None, kv=None, cache=None, q=None):
    kv = kv or case.handle()
    cache = cache or case.filled(kv)
    out, lse = kv.attention(cache, case.batch(), case.q.cuda() if q is None else q, window=window, sinks=sinks,
                            scale=scale)
    torch.cuda.synchronize()
    rc, word = kv.status()
    assert rc == B.MOE_FFN_OK, B.decode_status(word)
    want, wl, tol, ltol = attention(case, scale, window, sinks)
    check_close(lse, wl, ltol, "lse")
    check_close(out, want, tol, "out")
    return out, lse
