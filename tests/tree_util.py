"""Trees of drafted tokens for the paged cache's tests, and their attention by its definition in 64 bits, a row at a
time. The tolerances are those of tests/kv_util.py: what a row sees is another, what is done with it the same."""
import math

import torch

from tests.kv_util import BF, F32

SHAPES = ("random", "chain", "star", "roots", "binary", "comb")


def parents(shape, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [min(i, 1) - 1 for i in range(n)]
    if shape == "roots":
        return [-1] * n
    if shape == "binary":
        return [(i + 1) // 2 - 1 for i in range(n)]
    if shape == "comb":  # a chain of every other node, each with a leaf
        return [-1 if i == 0 else i - 2 if i % 2 == 0 else i - 1 for i in range(n)]
    return [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)]


def path_to(parent, i):
    """The nodes from the root down to i."""
    path = [i]
    while parent[path[0]] >= 0:
        path.insert(0, parent[path[0]])
    return path


def visible(case, parent, b, i, window, sinks):
    """Slots that node i of sequence b sees."""
    old = case.kv[b] - case.new[b]
    path = path_to(parent, i)
    p = old + len(path) - 1
    slots = list(range(old)) + [old + j for j in path]
    positions = list(range(old)) + [old + d for d in range(len(path))]
    return [s for s, at in zip(slots, positions) if window == 0 or at > p - window or at < sinks]


def attention(case, trees, window=0, sinks=0, scale=None):
    """(out, lse, tolerance of out, tolerance of lse)."""
    scale = case.d ** -0.5 if scale is None else scale
    out = torch.zeros(case.T, case.hq, case.d, dtype=torch.float64)
    lse = torch.full((case.T, case.hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    g = case.hq // case.hkv
    for b, n in enumerate(case.new):
        k, v = case.stored("k", b), case.stored("v", b)
        for i in range(n):
            row = case.cu[b] + i
            at = torch.tensor(visible(case, trees[b], b, i, window, sinks), dtype=torch.long)
            for h in range(case.hkv):
                hs = slice(h * g, (h + 1) * g)
                q, kk, vv = case.q[row, hs].double(), k[at, h], v[at, h]
                s = scale * q @ kk.T
                ds = case.d * F32 * scale * (q.abs() @ kk.abs().T) + 4 * F32 * s.abs()
                if case.fmt == "e4m3":
                    ds = ds + 2.0 ** -17 * scale * q.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)
                ds = ds.amax(-1, keepdim=True)
                w = torch.softmax(s, -1)
                out[row, hs], lse[row, hs] = w @ vv, torch.logsumexp(s, -1)
                rel = torch.expm1(2 * ds) + 2.0 ** -20 + BF + 2 * len(at) * F32
                tol[row, hs] = rel * (w @ vv.abs()) * (1 + BF) + BF * out[row, hs].abs()
                ltol[row, hs] = ds[:, 0] + 2.0 ** -20 + len(at) * F32 + 4 * F32 * lse[row, hs].abs()
    return out, lse, tol, ltol
