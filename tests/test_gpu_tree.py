"""Trees of drafted tokens over the paged cache on a GB300: their masks, their attention against its definition in 64
bits (tests/tree_util.py), the path that is kept, the beams that are reordered, and a run of the operators together."""
import importlib.util
import math
import os

import pytest
import torch

import tests.kv_util as U
import tests.tree_util as W
from mixture_experts_ffn_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 128), ("bf16", 256), ("bf16", 512), ("e4m3", 128), ("e4m3", 256), ("e4m3", 512)]
BAD = B.STATUS_BITS["BAD_INDEX"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def _ok(kv):
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_OK, 0)


def _flat(case, trees):
    p = [q for t in trees for q in t]
    return torch.tensor(p + [-5] * (case.T - len(p)), dtype=torch.int32).cuda()  # (rows of no sequence: anything)


def _trees(case, shape="random", seed=0):
    return [W.parents(shape, n, seed + b) for b, n in enumerate(case.new)]


def _check(case, trees, window=0, sinks=0, scale=None, kv=None, cache=None, q=None):
    kv = kv or case.handle()
    cache = cache or case.filled(kv)
    batch = case.batch()
    tree = kv.tree(batch, _flat(case, trees))
    q = case.q.cuda() if q is None else q
    out, lse = kv.tree_attention(cache, batch, tree, q, window=window, sinks=sinks, scale=scale,
                                 out=torch.full((case.T, case.hq, case.d), 7.0, dtype=torch.bfloat16, device="cuda"))
    _ok(kv)
    want, wl, tol, ltol = W.attention(case, trees, window, sinks, scale)
    U.check_close(lse, wl, ltol, "lse")
    U.check_close(out, want, tol, "out")
    return out, lse


# ------------------------------------------------------------------ masks

@pytest.mark.parametrize("shape", W.SHAPES)
def test_masks_and_depths(shape):
    case = U.Case("bf16", 1, 1, 128, 16, [1, 0, 31, 32, 33, 256, 2], [1, 5, 31, 40, 400, 300, 9], pad_rows=3)
    kv = case.handle()
    trees = _trees(case, shape)
    tree = kv.tree(case.batch(), _flat(case, trees))
    _ok(kv)
    masks, depth = tree.masks.cpu().tolist(), tree.depth.tolist()
    for b, t in enumerate(trees):
        for i in range(len(t)):
            path = W.path_to(t, i)
            bits = sum((w & 0xffffffff) << (32 * j) for j, w in enumerate(masks[case.cu[b] + i]))
            assert bits == sum(1 << j for j in path) and depth[case.cu[b] + i] == len(path) - 1
    assert not tree.masks[case.cu[-1]:].any() and not tree.depth[case.cu[-1]:].any()


def test_bad_parents_count_as_roots():
    case = U.Case("bf16", 2, 1, 128, 16, [5, 4], [20, 9], seed=1)
    kv = case.handle()
    cache = case.filled(kv)
    for bad in (-2, 2, 3, 2 ** 31 - 1, -2 ** 31):
        p = torch.tensor([-1, 0, bad, 1, 2, -1, 0, 1, 2], dtype=torch.int32, device="cuda")
        tree = kv.tree(case.batch(), p)
        torch.cuda.synchronize()
        assert kv.status() == (B.MOE_FFN_EDEVICE, BAD)
        p[2] = -1
        same = kv.tree(case.batch(), p)
        assert torch.equal(tree.masks, same.masks) and torch.equal(tree.depth, same.depth)
    _check(case, [[-1, 0, -1, 1, 2], [-1, 0, 1, 2]], kv=kv, cache=cache)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("shape", W.SHAPES)
def test_shapes_of_trees(fmt, d, shape):
    case = U.Case(fmt, 4, 2, d, 32, [12, 1, 40, 7], [33, 300, 40, 135], seed=d, pad_rows=2)
    _check(case, _trees(case, shape))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_where_contexts_end(fmt, page):
    """Contexts of 0 and 1 tokens, to page and tile borders and just over them."""
    old = [0, 1, page - 1, page, 127, 128, 129, 250]
    new = [9, 17, 1, 3, 2, 5, 128, 6]
    case = U.Case(fmt, 2, 1, 256, page, new, [a + b for a, b in zip(old, new)], seed=page)
    _check(case, _trees(case))


@pytest.mark.parametrize("fmt,d,group", [("bf16", 128, 1), ("bf16", 256, 3), ("e4m3", 256, 5), ("bf16", 512, 8), ("e4m3", 512, 16),
                                         ("bf16", 128, 64)])
def test_head_groups_and_large_trees(fmt, d, group):
    """Trees over several row tiles."""
    case = U.Case(fmt, group, 1, d, 16, [256 if group < 8 else 70, 3], [290, 40], seed=group)
    _check(case, _trees(case))


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (3, 0), (7, 4), (64, 0), (64, 200), (130, 7), (1000, 3)])
def test_windows_and_sinks(fmt, d, window, sinks):
    """Windows that end among the ancestors, sinks that lie among them, and both in the context."""
    case = U.Case(fmt, 2, 1, d, 16, [40, 33, 12], [340, 33, 13], seed=d + window)
    trees = [W.parents("chain", 40), W.parents("comb", 33), W.parents("random", 12, 3)]
    _check(case, trees, window, sinks)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(2 ** 40, 2 ** 40), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_windows_and_sinks_as_long_as_numbers_go(fmt, window, sinks):
    case = U.Case(fmt, 2, 1, 256, 16, [20, 6], [100, 6], seed=4)
    _check(case, _trees(case), window, sinks)


@pytest.mark.parametrize("fmt,hq,hkv,d,page,new,kv,window,sinks", [
    ("bf16", 16, 2, 512, 128, [16], [9000], 0, 0), ("e4m3", 16, 8, 256, 64, [24, 2, 9], [5000, 700, 130], 1024, 4),
    ("bf16", 8, 8, 128, 16, [64], [7001], 0, 0), ("e4m3", 12, 4, 128, 32, [5] * 20, [5 + 97 * i for i in range(20)], 0, 0)])
def test_long_caches(fmt, hq, hkv, d, page, new, kv, window, sinks):
    """Work split over a long context, and many sequences."""
    case = U.Case(fmt, hq, hkv, d, page, new, kv, seed=d)
    _check(case, _trees(case), window, sinks)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("hq,hkv,most", [(2, 2, 16), (3, 1, 5), (8, 4, 8), (16, 2, 2), (16, 1, 1), (12, 4, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2), (130, 0), (300, 140)])
def test_few_rows(d, hq, hkv, most, window, sinks):
    """At most 16 rows to a kv head, over pages of every size, contexts that end anywhere in a tile, empty sequences."""
    new = [most, 1, 0, max(1, most // 2), most, most, 1, most]
    kv = [most, 1, 17, 127, 128 + most, 700, 129, 1500]
    for page in (16, 64, 128):
        case = U.Case("e4m3", hq, hkv, d, page, new, kv, pad_rows=2, seed=page + most)
        for shape in ("random", "chain", "star"):
            _check(case, _trees(case, shape), window, sinks)


@pytest.mark.parametrize("d", [128, 256])
def test_few_rows_of_many_and_long_sequences(d):
    _check(*(lambda c: (c, _trees(c)))(U.Case("e4m3", 4, 2, d, 16, [2, 1, 8, 3] * 100, [9, 1, 150, 30] * 100, seed=d)))
    case = U.Case("e4m3", 2, 1, d, 64, [8], [40_000], seed=d + 1)  # its pieces are joined in groups
    _check(case, _trees(case))
    case = U.Case("e4m3", 4, 2, d, 128, [3, 4, 2], [9_000, 70, 20_000], seed=d + 2)
    _check(case, _trees(case), 8_000, 3)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_chain_is_the_causal_rule(fmt):
    case = U.Case(fmt, 8, 2, 256, 32, [30, 1, 64], [200, 50, 64], seed=6)
    kv = case.handle()
    cache = case.filled(kv)
    out, lse = _check(case, _trees(case, "chain"), kv=kv, cache=cache, window=20, sinks=3)
    causal, cl = kv.attention(cache, case.batch(), case.q.cuda(), window=20, sinks=3)
    _, _, tol, ltol = W.attention(case, _trees(case, "chain"), 20, 3)
    U.check_close(out, causal.double().cpu(), 2 * tol, "out")
    U.check_close(lse, cl.double().cpu(), 2 * ltol, "lse")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_trees_of_one_node(fmt):
    case = U.Case(fmt, 16, 2, 512, 64, [1] * 5, [1, 2, 70, 300, 64], seed=7)
    kv = case.handle()
    cache = case.filled(kv)
    out, lse = _check(case, [[-1]] * 5, kv=kv, cache=cache)
    want = kv.attention(cache, case.batch(), case.q.cuda())
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (4, 2), (40, 0)])
def test_hidden_values_do_not_matter(fmt, d, window, sinks):
    """A node whose keys and values are infinite or NaN reaches only those below it."""
    case = U.Case(fmt, 4, 2, d, 16, [20, 9], [150, 40], seed=d + window)
    trees = _trees(case, "comb")
    kv = case.handle()
    want, wl, tol, ltol = W.attention(case, trees, window, sinks)
    for name, value in (("k", math.nan), ("v", math.nan), ("v", -math.inf)):
        other = U.Case(fmt, 4, 2, d, 16, [20, 9], [150, 40], seed=d + window)
        for leaf in (3, 7, 19):  # leaves: seen by themselves alone
            getattr(other, name)[0][130 + leaf, :, 5] = value
        tree = kv.tree(other.batch(), _flat(other, trees))
        out, lse = kv.tree_attention(other.filled(kv), other.batch(), tree, other.q.cuda(), window=window, sinks=sinks)
        _ok(kv)
        seen = torch.zeros(other.T, dtype=torch.bool)
        seen[[3, 7, 19]] = True
        U.check_close(out[~seen.cuda()], want[~seen], tol[~seen], name)
        U.check_close(lse[~seen.cuda()], wl[~seen], ltol[~seen], name)
        assert not torch.isfinite(out[seen.cuda()]).all(-1).any()


def test_values_that_some_rows_see_come_back():
    """An infinite value high in the tree: all below it have it, in the row tiles of large trees too, others not."""
    case = U.Case("bf16", 2, 1, 256, 16, [250], [380], seed=8)
    trees = _trees(case, "random", 5)
    case.v[0][130 + 1, 0, 9] = math.inf
    kv = case.handle()
    tree = kv.tree(case.batch(), _flat(case, trees))
    out, _ = kv.tree_attention(case.filled(kv), case.batch(), tree, case.q.cuda())
    _ok(kv)
    below = torch.tensor([1 in W.path_to(trees[0], i) for i in range(250)])
    assert below.any() and not below.all()
    assert (out[below.cuda(), :, 9] == math.inf).all() and torch.isfinite(out[~below.cuda()]).all()
    assert torch.isfinite(out[..., :9]).all() and torch.isfinite(out[..., 10:]).all()


@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("big", [2.0 ** -30, 2.0 ** 30])
def test_values_of_far_apart_sizes(d, big):
    """e4m3 scales far apart, of nodes that only some rows see and of the context."""
    case = U.Case("e4m3", 4, 2, d, 16, [20, 4], [300, 200], seed=d)
    case.v[0][282] = (case.v[0][282].float() * big).to(torch.bfloat16)
    case.v[0][3] = (case.v[0][3].float() * big).to(torch.bfloat16)
    case.v[1][150:] = (case.v[1][150:].float() * big).to(torch.bfloat16)
    _check(case, _trees(case, "binary"))
    _check(case, _trees(case, "roots"), 60, 1)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4, 2), (40, 0)])
def test_few_rows_and_hidden_values(d, window, sinks):
    """As above, of up to 16 rows: what a node holds reaches only those below it, whatever its size, and bytes behind the
    last node reach nobody."""
    def case():
        return U.Case("e4m3", 4, 2, d, 16, [8, 5], [150, 40], seed=d + window)
    trees = _trees(case(), "comb")
    kv = case().handle()
    want, wl, tol, ltol = W.attention(case(), trees, window, sinks)
    for name, value in (("k", math.nan), ("k", math.inf), ("v", math.nan), ("v", -math.inf)):
        other = case()
        for leaf in (3, 7):  # leaves: seen by themselves alone
            getattr(other, name)[0][142 + leaf, :, 5] = value
        cache = other.filled(kv)
        for t in (cache.k, cache.v):  # the slots behind the second sequence's last node
            t.view(torch.uint8)[int(other.pages[1, 2]), :, 8:] = 0x7f
        for t in (cache.k_scale, cache.v_scale):
            t[int(other.pages[1, 2]), :, 8:] = math.nan
        tree = kv.tree(other.batch(), _flat(other, trees))
        out, lse = kv.tree_attention(cache, other.batch(), tree, other.q.cuda(), window=window, sinks=sinks)
        _ok(kv)
        seen = torch.zeros(other.T, dtype=torch.bool)
        seen[[3, 7]] = True
        U.check_close(out[~seen.cuda()], want[~seen], tol[~seen], name)
        U.check_close(lse[~seen.cuda()], wl[~seen], ltol[~seen], name)
        assert not torch.isfinite(out[seen.cuda()]).all(-1).any()
    for big in (2.0 ** -30, 2.0 ** 30):
        other = case()
        other.v[0][145] = (other.v[0][145].float() * big).to(torch.bfloat16)
        other.v[0][3] = (other.v[0][3].float() * big).to(torch.bfloat16)
        other.v[1][20:] = (other.v[1][20:].float() * big).to(torch.bfloat16)
        _check(other, _trees(other, "binary"), window, sinks)
        _check(other, _trees(other, "roots"), window, sinks)


def test_few_rows_captured_and_repeated():
    case = U.Case("e4m3", 8, 4, 256, 32, [8, 3, 8], [9000, 39, 600], seed=13)
    kv = case.handle()
    cache, batch = case.filled(kv), case.batch()
    p, q = _flat(case, _trees(case)), case.q.cuda()
    first = kv.tree_attention(cache, batch, kv.tree(batch, p), q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = kv.tree_attention(cache, batch, kv.tree(batch, p), q)
    for _ in range(5):
        graph.replay()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    for shape in ("chain", "star"):
        p.copy_(_flat(case, _trees(case, shape, 3)))
        graph.replay()
        _ok(kv)
        want, wl, tol, ltol = W.attention(case, _trees(case, shape, 3))
        U.check_close(out, want, tol, shape)
        U.check_close(lse, wl, ltol, shape)


def test_few_rows_with_bad_batches():
    """Sequences with more nodes than cached tokens, and pages that are none: status, and the others as they should be."""
    case = U.Case("e4m3", 4, 2, 128, 16, [4, 4, 4], [40, 40, 40], seed=14)
    kv = case.handle()
    cache = case.filled(kv)
    batch, q = case.batch(), case.q.cuda()
    tree = kv.tree(batch, _flat(case, _trees(case)))
    want = kv.tree_attention(cache, batch, tree, q)
    _ok(kv)
    short = batch.tensors[1].clone()
    short[1] = 3
    out, lse = kv.tree_attention(cache, B.KVBatch(batch.tensors[0], short, batch.tensors[2], max_new=4), tree, q)
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, BAD)
    assert (out[4:8] == 0).all() and (lse[4:8] == -math.inf).all()
    for i in (slice(0, 4), slice(8, 12)):
        assert torch.equal(out[i], want[0][i]) and torch.equal(lse[i], want[1][i])
    none = batch.tensors[2].clone()
    none[1, 0] = 10 ** 6
    out, lse = kv.tree_attention(cache, B.KVBatch(batch.tensors[0], batch.tensors[1], none, max_new=4), tree, q)
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, BAD)
    for i in (slice(0, 4), slice(8, 12)):
        assert torch.equal(out[i], want[0][i]) and torch.equal(lse[i], want[1][i])


def test_rows_far_apart_and_strided_queries():
    case = U.Case("bf16", 8, 2, 128, 32, [6, 9], [100, 9], seed=9)
    fused = torch.zeros(case.T, 12, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = case.q.cuda()
    _check(case, _trees(case), scale=0.3, q=fused[:, 2:10])


def test_batches_without_context_or_tokens():
    """A sequence with fewer cached tokens than nodes sees nothing, which is reported; the others do not notice."""
    case = U.Case("bf16", 4, 2, 256, 16, [4, 6, 3], [30, 6, 50], seed=10, pad_rows=1)
    kv = case.handle()
    cache = case.filled(kv)
    batch = case.batch()
    trees = _trees(case)
    want, _ = kv.tree_attention(cache, batch, kv.tree(batch, _flat(case, trees)), case.q.cuda())
    batch.tensors[1][1] = 5
    out, lse = kv.tree_attention(cache, batch, kv.tree(batch, _flat(case, trees)), case.q.cuda(),
                                 out=torch.ones_like(want))
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, BAD)
    assert not out[4:10].any() and (lse[4:10] == -math.inf).all()
    assert torch.equal(out[:4], want[:4]) and torch.equal(out[10:], want[10:])
    none = B.KVBatch(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                     torch.zeros(0, 1, dtype=torch.int32, device="cuda"), max_new=0)
    tree = kv.tree(none, torch.full((3,), 9, dtype=torch.int32, device="cuda"))
    assert not tree.masks.any() and not tree.depth.any()
    out, lse = kv.tree_attention(cache, none, tree, case.q.cuda()[:3])
    assert not out.any() and (lse == -math.inf).all()
    tree = kv.tree(none, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert kv.tree_attention(cache, none, tree, case.q.cuda()[:0])[0].shape == (0, 4, 256)
    _ok(kv)


def test_masks_that_say_too_much():
    """Bits after a node's own, of masks that kv.tree did not make, are not looked at."""
    case = U.Case("bf16", 4, 2, 256, 16, [10, 20], [40, 20], seed=11)
    kv = case.handle()
    cache = case.filled(kv)
    batch = case.batch()
    trees = _trees(case)
    tree = kv.tree(batch, _flat(case, trees))
    want = kv.tree_attention(cache, batch, tree, case.q.cuda())
    for b, n in enumerate(case.new):
        for i in range(n):
            for w in range(8):
                above = sum(1 << j for j in range(32) if 32 * w + j > i)
                tree.masks[case.cu[b] + i, w] |= above - (1 << 32) if above >= 1 << 31 else above
    out = kv.tree_attention(cache, batch, tree, case.q.cuda())
    _ok(kv)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_captured_tree_replays_with_new_trees():
    case = U.Case("bf16", 8, 2, 256, 32, [12, 7], [100, 39], seed=12)
    kv = case.handle()
    cache = case.filled(kv)
    batch = case.batch()
    p, q = _flat(case, _trees(case)), case.q.cuda()
    kv.tree_attention(cache, batch, kv.tree(batch, p), q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = kv.tree_attention(cache, batch, kv.tree(batch, p), q)
    for shape in ("chain", "star", "random"):
        p.copy_(_flat(case, _trees(case, shape, 3)))
        graph.replay()
        _ok(kv)
        want, wl, tol, ltol = W.attention(case, _trees(case, shape, 3))
        U.check_close(out, want, tol, shape)
        U.check_close(lse, wl, ltol, shape)


# ------------------------------------------------------------------ keep

def _bits(c):
    return {n: t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)
            for n, t in (("k", c.k), ("v", c.v), ("k_scale", c.k_scale), ("v_scale", c.v_scale)) if t is not None}


def _random_cache(kv, seed):
    """A cache of random bytes, but for scales, which are random numbers."""
    g = torch.Generator().manual_seed(seed)
    c = kv.new_cache()
    for n, t in _bits(c).items():
        t.copy_(torch.randint(-100 if t.dtype != torch.uint8 else 0, 100, t.shape, generator=g).to(t.dtype))
    return c


def _kept(case, cache, nodes, counts):
    want = {n: t.clone() for n, t in _bits(cache).items()}
    was = {n: t.clone() for n, t in want.items()}
    for b in range(len(case.new)):
        old = case.kv[b] - case.new[b]
        for i in range(counts[b]):
            src, dst = old + nodes[b][i], old + i
            sp, dp = int(case.pages[b, src // case.page]), int(case.pages[b, dst // case.page])
            for n in want:
                want[n][dp, :, dst % case.page] = was[n][sp, :, src % case.page]
    return want


def _table(rows, cols):
    return torch.tensor([list(r) + [-1] * (cols - len(r)) for r in rows], dtype=torch.int32).view(len(rows), cols).cuda()


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("page,hkv", [(16, 3), (128, 1), (32, 8)])
def test_kept_paths(fmt, d, page, hkv):
    new, kv_len = [1, 40, 256, 3, 0, 17], [5, 50, 300, 3, 20, 33]
    case = U.Case(fmt, hkv, hkv, d, page, new, kv_len, seed=page)
    kv = case.handle()
    rows = [[0], list(range(1, 40, 2)), list(range(0, 100)) + list(range(130, 256)), [2], [], [0, 1, 2, 16]]
    counts = [1, 20, 226, 1, 0, 3]
    layers = [_random_cache(kv, i) for i in range(3)]
    want = [_kept(case, c, rows, counts) for c in layers]
    left = kv.keep(layers, case.batch(), _table(rows, 230), torch.tensor(counts, dtype=torch.int32, device="cuda"))
    _ok(kv)
    assert left.tolist() == [k - n + c for k, n, c in zip(kv_len, new, counts)]
    for c, w in zip(layers, want):
        for n, t in _bits(c).items():
            assert torch.equal(t, w[n]), n


def test_many_layers_and_one():
    case = U.Case("e4m3", 2, 2, 128, 16, [9], [30], seed=1)
    kv = case.handle()
    counts = torch.tensor([2], dtype=torch.int32, device="cuda")
    layers = [_random_cache(kv, i) for i in range(70)]
    want = [_kept(case, c, [[4, 8]], [2]) for c in layers]
    assert kv.keep(layers, case.batch(), _table([[4, 8]], 2), counts).tolist() == [23]
    for c, w in zip(layers, want):
        assert all(torch.equal(t, w[n]) for n, t in _bits(c).items())
    one = _random_cache(kv, 5)
    kv.keep(one, case.batch(), _table([[4, 8]], 2), counts)
    assert all(torch.equal(t, want[5][n]) for n, t in _bits(one).items())
    _ok(kv)


@pytest.mark.parametrize("path,count,moved", [([0, 5, 4], 3, 2), ([0, 0], 2, 1), ([1, 12], 2, 1), ([-1, 3], 2, 0), ([3, 4], 3, 2),
                                              ([3, 4], -1, 0), ([0, 1, 1, 7], 4, 2), ([2 ** 31 - 1, 3], 2, 0)])
def test_bad_paths_stop_and_are_reported(path, count, moved):
    case = U.Case("bf16", 2, 2, 128, 16, [12, 12], [30, 40], seed=2)
    kv = case.handle()
    c = _random_cache(kv, 3)
    want = _kept(case, c, [path, [3, 9]], [moved, 2])
    rows = _table([path, [3, 9]], len(path))
    left = kv.keep(c, case.batch(), rows, torch.tensor([count, 2], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, BAD)
    assert left.tolist() == [18 + moved, 30]
    assert all(torch.equal(t, want[n]) for n, t in _bits(c).items())


def test_keep_with_bad_tables_touches_nothing_else():
    case = U.Case("bf16", 2, 2, 128, 16, [12, 12], [30, 40], seed=2)
    kv = case.handle()
    counts = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    for change in ("page", "short"):
        c = _random_cache(kv, 3)
        batch = case.batch()
        if change == "page":
            batch.tensors[2][0, 1] = -1  # positions 16 to 31: both nodes of the first path
        else:
            batch.tensors[1][0] = 11
        want = _kept(case, c, [[], [3, 9]], [0, 2])
        left = kv.keep(c, batch, _table([[3, 9], [3, 9]], 2), counts)
        torch.cuda.synchronize()
        assert kv.status() == (B.MOE_FFN_EDEVICE, BAD), change
        assert left.tolist()[1] == 30 and (change == "page" or left.tolist()[0] == 11)
        assert all(torch.equal(t, want[n]) for n, t in _bits(c).items()), change


# ------------------------------------------------------------------ reorder

def _beams(users, beams, page, lengths, seed=0, spare=2):
    """A page table whose beams share full pages by chance and own those from the one under way on."""
    g = torch.Generator().manual_seed(seed)
    cols = max(n // page for n in lengths) + spare
    n_pages = sum(n // page for n in lengths) * 2 + users * beams * cols + 3
    order = torch.randperm(n_pages, generator=g).tolist()
    rows = []
    for u in range(users):
        full = lengths[u] // page
        shared = [[order.pop(), order.pop()] for _ in range(full)]
        for _ in range(beams):
            pick = torch.randint(0, 2, (max(full, 1),), generator=g).tolist()
            rows.append([s[i] for s, i in zip(shared, pick)] + [order.pop() for _ in range(cols - full)])
    return torch.tensor(rows, dtype=torch.int32), n_pages


def _reordered(table, lengths, parents, page, layers):
    users, beams = len(parents), len(parents[0])
    want_table = table.clone()
    want = [{n: t.clone() for n, t in _bits(c).items()} for c in layers]
    for u in range(users):
        full, rest = divmod(lengths[u], page)
        for k in range(beams):
            me, of = u * beams + k, u * beams + parents[u][k]
            want_table[me, :full] = table[of, :full]
            if rest:
                for w, c in zip(want, layers):
                    for n, t in _bits(c).items():
                        w[n][int(table[me, full]), :, :rest] = t[int(table[of, full]), :, :rest]
    return want_table, want


@pytest.mark.parametrize("fmt,d", SHAPES)
@pytest.mark.parametrize("page,hkv,beams", [(16, 3, 1), (16, 2, 2), (32, 8, 5), (64, 1, 8), (128, 2, 9), (16, 1, 64)])
def test_reordered_beams(fmt, d, page, hkv, beams):
    lengths = [0, 1, page - 1, page, 3 * page + page // 2]
    users = len(lengths)
    table, n_pages = _beams(users, beams, page, lengths, seed=beams)
    kv = B.PagedKV(hkv, hkv, d, page, n_pages, fmt, max_seqs=users * beams)
    layers = [_random_cache(kv, i) for i in range(2)]
    g = torch.Generator().manual_seed(page)
    parents = torch.randint(0, beams, (users, beams), generator=g)
    parents[4] = torch.randperm(beams, generator=g)
    parents[2] = beams - 1 - torch.arange(beams)
    want_table, want = _reordered(table, lengths, parents.tolist(), page, layers)
    wide = torch.full((users * beams, table.shape[1] + 3), -9, dtype=torch.int32, device="cuda")
    pages = wide[:, :table.shape[1]]
    pages.copy_(table)
    kv.reorder(layers, pages, torch.tensor(lengths, dtype=torch.int32, device="cuda"), parents.to(torch.int32).cuda())
    _ok(kv)
    assert torch.equal(pages.cpu(), want_table) and (wide[:, table.shape[1]:] == -9).all()
    for c, w in zip(layers, want):
        for n, t in _bits(c).items():
            assert torch.equal(t, w[n]), n


@pytest.mark.parametrize("n_layers", [0, 1, 40])
def test_reordered_layers(n_layers):
    lengths, parents = [37], [[2, 0, 1, 1]]
    table, n_pages = _beams(1, 4, 16, lengths)
    kv = B.PagedKV(2, 2, 128, 16, n_pages, "e4m3", max_seqs=4)
    layers = [_random_cache(kv, i) for i in range(n_layers)]
    want_table, want = _reordered(table, lengths, parents, 16, layers)
    pages = table.cuda()
    kv.reorder(layers, pages, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
               torch.tensor(parents, dtype=torch.int32, device="cuda"))
    _ok(kv)
    assert torch.equal(pages.cpu(), want_table)
    for c, w in zip(layers, want):
        assert all(torch.equal(t, w[n]) for n, t in _bits(c).items())


def test_bad_beams_are_reported():
    """Parents, lengths and page ids out of range: what is in range moves, nothing else is touched."""
    lengths = [37, 20]
    table, n_pages = _beams(2, 3, 16, lengths)
    kv = B.PagedKV(2, 2, 128, 16, n_pages, "bf16", max_seqs=6)
    parents = [[1, 1, 0], [0, 0, 0]]
    for change in ("parent", "negative", "length", "page"):
        c = _random_cache(kv, 1)
        n, p, t = list(lengths), [list(r) for r in parents], table.clone()
        if change == "parent":
            p[0][2] = 3
            good = [[1, 1, 2], [0, 0, 0]]
        elif change == "negative":
            p[0][0] = -1
            good = [[0, 1, 0], [0, 0, 0]]
        else:
            good = parents
        if change == "length":
            n[1] = -4
        want_table, want = _reordered(t, [37, 0] if change == "length" else lengths, good, 16, [c])
        if change == "page":
            t[4, 1] = n_pages  # beam 1 of user 1's page under way
            want_table[4, 1] = n_pages
            keep = int(table[4, 1])
            for name, x in _bits(c).items():
                want[0][name][keep] = x[keep]
        pages = t.cuda()
        kv.reorder(c, pages, torch.tensor(n, dtype=torch.int32, device="cuda"), torch.tensor(p, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert kv.status() == (B.MOE_FFN_EDEVICE, BAD), change
        assert torch.equal(pages.cpu(), want_table), change
        assert all(torch.equal(x, want[0][name]) for name, x in _bits(c).items()), change


def test_captured_moves():
    case = U.Case("bf16", 2, 2, 128, 16, [6], [30], seed=2)
    kv = case.handle()
    c = _random_cache(kv, 1)
    batch, nodes = case.batch(), _table([[2, 5]], 2)
    counts = torch.tensor([2], dtype=torch.int32, device="cuda")
    start = {n: t.clone() for n, t in _bits(c).items()}
    kv.keep(c, batch, nodes, counts)
    table, _ = _beams(1, 2, 16, [5], spare=1)
    pages = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    length, parents = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([5], [[0, 0]]))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    two = B.PagedKV(2, 2, 128, 16, case.n_pages, "bf16", max_seqs=2)
    other = two.new_cache()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        left = kv.keep(c, batch, nodes, counts)
        two.reorder(other, pages, length, parents)
    for n, t in _bits(c).items():
        t.copy_(start[n])
    other.k.normal_()
    nodes.copy_(_table([[1, 3]], 2))
    want = _kept(case, c, [[1, 3]], [2])
    graph.replay()
    _ok(kv)
    assert left.tolist() == [26] and all(torch.equal(t, want[n]) for n, t in _bits(c).items())
    assert torch.equal(other.k[1, :, :5], other.k[0, :, :5]) and not torch.equal(other.k[1, :, 5:], other.k[0, :, 5:])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("layer,fmt", [("sliding", "bf16"), ("global", "e4m3")])
def test_example_drafts_and_searches(layer, fmt, capsys):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")
    spec = importlib.util.spec_from_file_location("serve_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off, status = m.main(["--layer", layer, "--format", fmt, "--users", "3", "--steps", "4", "--draft", "9", "--beams", "3"])
    assert off < 2e-2 and status == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_drafted_path_is_what_its_tokens_give_one_by_one(fmt):
    """A tree's tokens written, attended to and one path kept: each node of it got what the same tokens get as plain new
    ones, and the cache that remains holds them."""
    case = U.Case(fmt, 8, 2, 256, 16, [14, 14, 14], [60, 14, 131], seed=20)
    kv = case.handle()
    cache = case.filled(kv)
    trees = _trees(case, "random", 8)
    batch = case.batch()
    q = case.q.cuda()
    out, lse = kv.tree_attention(cache, batch, kv.tree(batch, _flat(case, trees)), q, window=40, sinks=2)
    _, _, tol, ltol = W.attention(case, trees, 40, 2)
    paths = [W.path_to(t, max(range(14), key=lambda i: len(W.path_to(t, i)))) for t in trees]
    longest = max(len(p) for p in paths)
    left = kv.keep(cache, batch, _table(paths, longest), torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"))
    rows = torch.tensor([case.cu[b] + i for b, p in enumerate(paths) for i in p]).cuda()
    cu = torch.tensor([0] + [len(p) for p in paths], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    chain = B.KVBatch(cu, left, case.pages.cuda(), max_new=longest)
    plain, pl = kv.attention(cache, chain, q[rows], window=40, sinks=2)
    _ok(kv)
    assert left.tolist() == [k - 14 + len(p) for k, p in zip(case.kv, paths)]
    U.check_close(out[rows], plain.double().cpu(), 2 * tol[rows.cpu()], "out")
    U.check_close(lse[rows], pl.double().cpu(), 2 * ltol[rows.cpu()], "lse")


# ------------------------------------------------------------------ refusals

def test_refusals():
    case = U.Case("e4m3", 4, 2, 256, 16, [5, 5], [20, 30], seed=30)
    kv = case.handle()
    cache = case.filled(kv)
    batch, q = case.batch(), case.q.cuda()
    p = _flat(case, _trees(case))
    tree = kv.tree(batch, p)
    counts, nodes = torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for call, match in ((lambda: kv.tree(batch, p.long()), "parents"), (lambda: kv.tree(batch, p.view(2, 5)), "parents"),
                        (lambda: kv.tree(batch, p.cpu()), "parents"), (lambda: kv.tree_attention(cache, batch, tree, q[:9]), "tokens"),
                        (lambda: kv.keep(cache, batch, nodes, counts[:1]), "counts"),
                        (lambda: kv.keep(cache, batch, nodes.view(-1), counts), "nodes"),
                        (lambda: kv.keep(cache, batch, nodes.long(), counts), "nodes"),
                        (lambda: kv.keep(dict(k=cache.k, v=cache.v), batch, nodes, counts), "k_scale"),
                        (lambda: kv.reorder(cache, batch.tensors[2], counts, nodes[:1]), "lengths"),
                        (lambda: kv.reorder(cache, batch.tensors[2].long(), counts, nodes), "pages"),
                        (lambda: kv.reorder(cache, batch.tensors[2].T.contiguous().T, counts, nodes), "pages")):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(B.MoeFFNError):  # more nodes than a tree has
        kv.tree(B.KVBatch(*batch.tensors, max_new=257), p)
    with pytest.raises(B.MoeFFNError):
        kv.tree_attention(cache, B.KVBatch(*batch.tensors, max_new=257), tree, q)
    with pytest.raises(B.MoeFFNError):
        kv.keep([], batch, nodes, counts)
    with pytest.raises(B.MoeFFNError):  # more beams than the handle has sequences
        kv.reorder(cache, torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                   torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(B.MoeFFNError):
        kv.tree_attention(cache, batch, tree, q, scale=-1.0)
    with pytest.raises(B.MoeFFNError):
        kv.tree_attention(cache, batch, tree, q, out=q)
    masks = torch.zeros(10 * 4 * 256 * 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(B.MoeFFNError):  # the masks in the output
        kv.tree_attention(cache, batch, B.KVTree(masks[:320].view(torch.int32).view(10, 8), tree.depth), q,
                          out=masks.view(torch.bfloat16).view(10, 4, 256))
    kv.close()
    for call in (lambda: kv.tree(batch, p), lambda: kv.tree_attention(cache, batch, tree, q),
                 lambda: kv.keep(cache, batch, nodes, counts)):
        with pytest.raises(B.MoeFFNError):
            call()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_caches_given_twice_are_refused(fmt):
    case = U.Case(fmt, 2, 2, 128, 16, [4, 5], [20, 30], seed=31)
    kv = case.handle()
    a, b = _random_cache(kv, 1), _random_cache(kv, 2)
    was = {n: t.clone() for n, t in _bits(a).items()}
    batch, counts = case.batch(), torch.ones(2, dtype=torch.int32, device="cuda")
    nodes = torch.full((2, 1), 3, dtype=torch.int32, device="cuda")
    scales = dict(k_scale=a.k_scale, v_scale=a.v_scale) if fmt == "e4m3" else {}
    lists = [[a, b, a], [a, dict(k=b.k, v=a.k, **scales)], [dict(k=a.k, v=a.k, **scales)]]
    if fmt == "e4m3":
        lists += [[dict(k=a.k, v=a.v, k_scale=a.k_scale, v_scale=a.k_scale)],
                  [b, dict(k=a.k, v=a.v, k_scale=a.k_scale, v_scale=b.k_scale)]]
    for caches in lists:
        with pytest.raises(B.MoeFFNError):
            kv.keep(caches, batch, nodes, counts)
        with pytest.raises(B.MoeFFNError):
            kv.reorder(caches, batch.tensors[2].contiguous(), torch.full((1,), 5, dtype=torch.int32, device="cuda"),
                       torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"))
    _ok(kv)
    assert all(torch.equal(t, was[n]) for n, t in _bits(a).items())


def test_moves_past_32_bits():
    hkv, d, page, n_pages = 8, 512, 64, 8448  # 2.2e9 elements
    kv = B.PagedKV(hkv, hkv, d, page, n_pages, "bf16", max_tokens=64, max_seqs=2)
    c = kv.new_cache()
    last = [n_pages - 1, n_pages - 2, n_pages - 3, n_pages - 4]
    g = torch.Generator(device="cuda").manual_seed(3)
    for p in last:
        c.k[p] = torch.randn(hkv, page, d, generator=g, device="cuda").to(torch.bfloat16)
        c.v[p] = torch.randn(hkv, page, d, generator=g, device="cuda").to(torch.bfloat16)
    pages = torch.tensor([last[:2], last[2:]], dtype=torch.int32, device="cuda")
    want = {n: t[last].clone() for n, t in (("k", c.k), ("v", c.v))}
    # Beams at 70 tokens change places: 6 slots of their second pages, and the tables' first entries.
    kv.reorder(c, pages, torch.tensor([70], dtype=torch.int32, device="cuda"),
               torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"))
    assert pages.tolist() == [[last[2], last[1]], [last[0], last[3]]]
    for w in want.values():
        w[1, :, :6], w[3, :, :6] = w[3, :, :6].clone(), w[1, :, :6].clone()
    # Of trees of ten nodes in the slots from 60 on, nodes 2, 5 and 9 stay.
    batch = B.KVBatch(torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"),
                      torch.tensor([70, 70], dtype=torch.int32, device="cuda"), pages, max_new=10)
    left = kv.keep(c, batch, torch.tensor([[2, 5, 9]] * 2, dtype=torch.int32, device="cuda"),
                   torch.tensor([3, 3], dtype=torch.int32, device="cuda"))
    assert left.tolist() == [63, 63]
    for w in want.values():
        for first, second in ((2, 1), (0, 3)):
            w[first, :, 60], w[first, :, 61], w[first, :, 62] = w[first, :, 62].clone(), w[second, :, 1].clone(), w[second, :, 5].clone()
    _ok(kv)
    for n, t in (("k", c.k), ("v", c.v)):
        assert torch.equal(t[last], want[n]), n
        assert not t[:n_pages - 4].any(), n


@pytest.mark.parametrize("fmt,beams", [("bf16", 3), ("e4m3", 20)])
def test_reordered_pages_of_many_rows(fmt, beams):
    """More rows to a block than it has threads."""
    page, lengths = 128, [127, 100, 255, 129, 128, 60] * 3
    table, n_pages = _beams(len(lengths), beams, page, lengths, seed=beams)
    kv = B.PagedKV(8, 8, 256, page, n_pages, fmt, max_seqs=len(lengths) * beams)
    layers = [_random_cache(kv, i) for i in range(2)]
    parents = torch.randint(0, beams, (len(lengths), beams), generator=torch.Generator().manual_seed(beams))
    want_table, want = _reordered(table, lengths, parents.tolist(), page, layers)
    pages = table.cuda()
    kv.reorder(layers, pages, torch.tensor(lengths, dtype=torch.int32, device="cuda"), parents.to(torch.int32).cuda())
    _ok(kv)
    assert torch.equal(pages.cpu(), want_table)
    for c, w in zip(layers, want):
        assert all(torch.equal(t, w[n]) for n, t in _bits(c).items())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq", [2, 8, 16, 24])
def test_single_nodes_without_room_are_reported(fmt, hq):
    """A sequence of one node of which the cache holds nothing, whichever kernel takes the batch."""
    case = U.Case(fmt, hq, 1, 128, 16, [1, 1, 1], [30, 1, 50], seed=12)
    kv = case.handle()
    cache = case.filled(kv)
    batch = case.batch()
    tree = kv.tree(batch, torch.full((3,), -1, dtype=torch.int32, device="cuda"))
    want, want_lse = kv.tree_attention(cache, batch, tree, case.q.cuda())
    _ok(kv)
    batch.tensors[1][1] = 0
    out, lse = kv.tree_attention(cache, batch, tree, case.q.cuda(), out=torch.ones_like(want))
    torch.cuda.synchronize()
    assert kv.status() == (B.MOE_FFN_EDEVICE, BAD)
    assert not out[1].any() and (lse[1] == -math.inf).all()
    assert torch.equal(out[::2], want[::2]) and torch.equal(lse[::2], want_lse[::2])
    # Of tokens that are no tree the same is no error.
    kv.attention(cache, batch, case.q.cuda())
    _ok(kv)


def test_a_tree_dropped_while_another_stream_still_attends():
    """The memory of its masks goes to new tensors of the stream that made them only after the queued attention."""
    case = U.Case("bf16", 4, 2, 256, 16, [10, 20], [40, 50], seed=14)
    kv = case.handle()
    cache = case.filled(kv)
    batch = case.batch()
    q, parents = case.q.cuda(), _flat(case, _trees(case))
    want, _ = kv.tree_attention(cache, batch, kv.tree(batch, parents), q)
    large = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    tree = kv.tree(batch, parents)
    nbytes = tree.masks.numel() * 4
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(40):
            large.fill_(i)
        got, _ = kv.tree_attention(cache, batch, tree, q)
    del tree
    over = [torch.zeros(nbytes, dtype=torch.uint8, device="cuda") for _ in range(200)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(over) == 200
    _ok(kv)
